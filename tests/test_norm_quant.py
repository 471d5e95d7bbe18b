"""The residual norm (forward, backward, 8-bit rows) and the row quantiser."""
import ctypes

import numpy as np
import pytest
import torch

from lowbit_util import U, gamma, half_step, rows_to_8bit
from mixture_experts_projections_b200 import rom

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
FAKE = 1 << 20  # 16-byte aligned, never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_projections_b200.build import build
    build()
    return rom.load_library()


# ------------------------------------------------------------------ refusals (no GPU)


def far(i):
    return ctypes.c_void_p(FAKE + i * (1 << 32))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(res_dtype=5), 1), (dict(T=-1), 1), (dict(Dm=0), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(y_scale=None), 1), (dict(y8=None), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(res_out=None, y=None, y8=None, y_scale=None, rstd=None), 1),
    (dict(dtype=0, res_dtype=1), 2), (dict(Dm=12), 2), (dict(Dm=16392), 2), (dict(T=1 << 31), 2),
    (dict(x=ctypes.c_void_p(FAKE + 2)), 2), (dict(w=ctypes.c_void_p(FAKE + 4)), 2),
    (dict(y8=ctypes.c_void_p(FAKE + 8)), 2),
    # overlaps: y8 in x, rstd in y, res_out half over res
    (dict(y8=far(0)), 1), (dict(rstd=far(4)), 1), (dict(res_out=ctypes.c_void_p(FAKE + (1 << 32) + 16)), 1),
])
def test_add_rmsnorm_rejects_bad_arguments(lib, kw, code):
    a = dict(x=far(0), dtype=1, res=far(1), res_dtype=0, T=10, Dm=64, w=far(2), eps=1e-5,
             res_out=far(3), y=far(4), y8=far(5), y_scale=far(6), rstd=far(7), stream=None)
    a.update(kw)
    assert lib.rom_add_rmsnorm(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 1), (dict(T=-1), 1), (dict(Dm=-8), 1), (dict(dx=None, dres=None, dw=None), 1),
    (dict(dy=None), 1), (dict(res_out=None), 1), (dict(rstd=None), 1),
    (dict(dtype=0, res_dtype=1), 2), (dict(Dm=20), 2), (dict(dx=ctypes.c_void_p(FAKE + 4)), 2),
    (dict(ws=None), 3), (dict(ws_bytes=64 * 4 * 10 - 1), 3),
    (dict(dx=far(0)), 1), (dict(dres=far(2)), 1), (dict(ws=far(3)), 1),
])
def test_add_rmsnorm_bwd_rejects_bad_arguments(lib, kw, code):
    a = dict(dy=far(0), dtype=1, dres_out=far(1), res_out=far(2), res_dtype=1, T=10, Dm=64,
             w=far(3), rstd=far(4), dx=far(5), dres=far(6), dw=far(7), ws=far(8),
             ws_bytes=64 * 4 * 10, stream=None)
    a.update(kw)
    assert lib.rom_add_rmsnorm_bwd(*a.values()) == code


def test_add_rmsnorm_bwd_workspace_size(lib):
    assert lib.rom_add_rmsnorm_bwd_workspace_size(0, 64) == 0
    assert lib.rom_add_rmsnorm_bwd_workspace_size(5, 0) == 0
    assert lib.rom_add_rmsnorm_bwd_workspace_size(5, 64) == 5 * 64 * 4
    assert lib.rom_add_rmsnorm_bwd_workspace_size(1 << 20, 64) == 512 * 64 * 4


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(K=0), 1), (dict(x=None), 1), (dict(scale=None), 1),
    (dict(K=12), 2), (dict(K=16392), 2), (dict(q=ctypes.c_void_p(FAKE + 8)), 2), (dict(q=far(0)), 1),
])
def test_quant_rows_rejects_bad_arguments(lib, kw, code):
    a = dict(x=far(0), dtype=1, rows=10, K=64, q=far(1), scale=far(2), stream=None)
    a.update(kw)
    assert lib.rom_quant_rows(*a.values()) == code


def test_binding_refuses_cpu_and_wrong_types():
    x = torch.zeros(4, 64, dtype=BF16)
    w = torch.ones(64)
    with pytest.raises(rom.RomError, match="contiguous CUDA"):
        rom.rom_add_rmsnorm(x, None, w, 1e-5, None, x.clone())
    with pytest.raises(rom.RomError, match="unsupported dtype"):
        rom.rom_add_rmsnorm(x.half(), None, w, 1e-5, None, None)
    with pytest.raises(rom.RomError, match="contiguous CUDA"):
        rom.rom_quant_rows(x, torch.zeros(4, 64, dtype=E4M3), torch.zeros(4))


# ------------------------------------------------------------------ numerics

# Longest chain of float32 roundings of a row's sum: up to 4 steps of 8
# elements per thread, 5 shuffles, 16 warps.
CHAIN = 4 * 8 + 5 + 16

gpu = pytest.mark.gpu


def make_rows(T, D, dtype, rt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, D, generator=g) * scale).to(dtype)
    res = (torch.randn(T, D, generator=g) * (1 + 2 * torch.randn(D, generator=g).abs()) * scale).to(rt)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    return x, res, w


def check_norm(x, res, w, eps, out, label):
    """Outputs (CPU) of the forward against the formula in 64 bits."""
    rt = out["res_out"].dtype
    s = x.float() if res is None else x.float() + res.float()  # one rounding, as the kernel's
    s = s.to(rt)
    assert torch.equal(out["res_out"], s), label
    s = s.double()
    D = s.shape[1]
    rstd = (s.square().mean(-1) + eps).rsqrt()
    # the sum's relative error is at most gamma(CHAIN), halved by the root; one
    # division and one addition, and rsqrtf's 2 ulp (4 U)
    r_rel = gamma(CHAIN) / 2 + 2 * U + 4 * U
    assert ((out["rstd"].double() - rstd).abs() <= r_rel * rstd).all(), label
    y = s * rstd[:, None] * w.double()
    y_rel = r_rel + 2 * U  # two products
    h = half_step(out["y"].dtype)
    tiny = torch.finfo(out["y"].dtype).tiny
    assert ((out["y"].double() - y).abs() <= (y_rel * (1 + h) + h) * y.abs() + tiny).all(), label
    if out.get("y8") is not None:
        a = y.abs().amax(-1).clamp(min=2.0 ** -100)
        sc = out["y_scale"].double()
        assert ((sc - a / 448).abs() <= (y_rel + U) * a / 448).all(), label
        v = out["y8"].double() * sc[:, None]
        # half a step of e4m3 (2^-4 of the value, 2^-10 codes among its
        # subnormals), and the float32 errors of y, of the factor and its product
        h8 = half_step(E4M3)
        assert ((v - y).abs() <= (h8 + 2 * (y_rel + 3 * U)) * y.abs() + 2.0 ** -10 * sc[:, None]).all(), label


def run_norm(x, res, w, eps, rt, q8=True):
    n = rom.add_rmsnorm(x.cuda(), None if res is None else res.cuda(), w.cuda(), eps, q8, rt)
    torch.cuda.synchronize()
    return dict(res_out=n.residual.cpu(), y=n.y.cpu(), rstd=n.rstd.cpu(),
                y8=None if n.y8 is None else n.y8.cpu(),
                y_scale=None if n.y_scale is None else n.y_scale.cpu())


@gpu
@pytest.mark.parametrize("D", [8, 64, 72, 128, 136, 248, 256, 264, 512, 520, 1000, 2048, 4096, 4104, 8192, 16384])
@pytest.mark.parametrize("dtype,rt", [(BF16, F32), (BF16, BF16), (F32, F32)])
def test_add_rmsnorm_matches_the_formula(D, dtype, rt):
    for T in (1, 9, 67):
        x, res, w = make_rows(T, D, dtype, rt, seed=D + T)
        check_norm(x, res, w, 1e-5, run_norm(x, res, w, 1e-5, rt), f"D={D} T={T}")


@gpu
def test_add_rmsnorm_without_residual_or_parts_of_the_outputs():
    x, _, w = make_rows(33, 264, BF16, F32, seed=1)
    check_norm(x, None, w, 1e-6, run_norm(x, None, w, 1e-6, F32), "no residual")
    full = run_norm(x, None, w, 1e-6, BF16)
    xd, wd = x.cuda(), w.cuda()
    y = torch.empty_like(xd)
    rom.rom_add_rmsnorm(xd, None, wd, 1e-6, None, y)  # residual type float32: s not rounded
    ro = torch.empty_like(xd)
    rom.rom_add_rmsnorm(xd, None, wd, 1e-6, ro, None)
    y8, sc = torch.empty(33, 264, dtype=E4M3, device="cuda"), torch.empty(33, device="cuda")
    rom.rom_add_rmsnorm(xd, None, wd, 1e-6, None, None, y8, sc)
    assert torch.equal(y.cpu(), full["y"]) and torch.equal(ro.cpu(), full["res_out"])
    assert torch.equal(y8.cpu().view(torch.uint8), full["y8"].view(torch.uint8))
    assert torch.equal(sc.cpu(), full["y_scale"])


@gpu
def test_add_rmsnorm_in_place_and_rows_do_not_depend_on_the_batch():
    for D, rt in ((264, F32), (2048, BF16), (8192, F32)):
        x, res, w = make_rows(300, D, BF16, rt, seed=D)
        ref = run_norm(x, res, w, 1e-5, rt)
        xd, rd = x.cuda(), res.cuda()
        rom.rom_add_rmsnorm(xd, rd, w.cuda(), 1e-5, rd, xd)
        assert torch.equal(rd.cpu(), ref["res_out"]) and torch.equal(xd.cpu(), ref["y"])
        one = run_norm(x[17:18], res[17:18], w, 1e-5, rt)
        for n in ("res_out", "y", "rstd", "y_scale"):
            assert torch.equal(one[n][0], ref[n][17]), n


@gpu
def test_add_rmsnorm_special_rows():
    """Rows of zeros, of tiny and of large values, and rows with NaN or infinity."""
    D = 520
    x = torch.zeros(7, D)
    x[1] = 1e-38 * torch.randn(D)
    x[2] = 1e17 * torch.randn(D)
    x[3] = torch.randn(D)
    x[3, 5] = float("nan")
    x[4] = torch.randn(D)
    x[4, 511] = float("inf")
    x[5, 0] = 1.0
    x[6] = torch.randn(D)
    w = torch.ones(D)
    out = run_norm(x, None, w, 1e-5, F32)
    fine = [0, 1, 2, 5, 6]
    check_norm(x[fine], None, w, 1e-5, {n: v[fine] for n, v in out.items()}, "special")
    assert (out["y8"][0].float() == 0).all() and out["y_scale"][0] == np.float32(2.0 ** -100) / np.float32(448)
    assert out["y"][3].isnan().all() and out["y8"][3].float().isnan().all() and out["y_scale"][3].isnan()
    # inf * rstd(inf) = inf * 0: NaN there, zeros elsewhere; no scale for the row
    assert out["y"][4, 511].isnan() and (out["y"][4, :511] == 0).all()
    assert out["y8"][4].float().isnan().all() and out["y_scale"][4].isnan()


def bwd_reference(dy, dres, s, w, rstd):
    dy, s, w, r = dy.double(), s.double(), w.double(), rstd.double()[:, None]
    D = s.shape[1]
    g = dy * w
    dot = (g * s).sum(-1, keepdim=True)
    d = 0 if dres is None else dres.double()
    ds = d + r * (g - s * r.square() * dot / D)
    # bounds: the dot's chain; the products around it, each a rounding of its
    # own operand
    dot_err = gamma(CHAIN + 2) * (g * s).abs().sum(-1, keepdim=True)
    k_err = r.square() / D * (dot_err + 5 * U * dot.abs())
    err = r * s.abs() * k_err + 6 * U * ((0 if dres is None else d.abs()) + r * g.abs() +
                                         r * s.abs() * r.square() * dot.abs() / D)
    dw = (dy * s * r).sum(0)
    T = s.shape[0]
    # a CTA's rows (148 of them or more, or one row each), 64 parts per warp, 8
    # warps, and two products
    n = -(-T // min(T, 148)) + 64 + 8 + 2
    return ds, err, dw, gamma(n) * (dy * s * r).abs().sum(0)


@gpu
@pytest.mark.parametrize("T,D", [(1, 8), (1, 16384), (3, 264), (37, 1000), (700, 64), (517, 1024),
                                 (600, 4104), (64, 8200), (500, 8200), (515, 56), (70, 72), (333, 128), (9, 136), (1203, 1536), (1001, 2048)])
@pytest.mark.parametrize("dtype,rt", [(BF16, F32), (BF16, BF16), (F32, F32)])
def test_add_rmsnorm_bwd_matches_the_formula(T, D, dtype, rt):
    dy, dres, w = make_rows(T, D, dtype, rt, seed=T + D)
    _, s, _ = make_rows(T, D, dtype, rt, seed=T + D + 1)
    rstd = (s.double().square().mean(-1) + 1e-5).rsqrt().float()
    d = [t.cuda() for t in (dy, dres, s, w, rstd)]
    for with_dres in (True, False):
        dx = torch.empty_like(d[0])
        dr = torch.empty_like(d[2])
        dw = torch.full((D,), float("nan"), device="cuda")
        ws = torch.full((rom.rom_add_rmsnorm_bwd_workspace_size(T, D) // 4,), float("nan"), device="cuda")
        rom.rom_add_rmsnorm_bwd(d[0], d[1] if with_dres else None, d[2], d[3], d[4], dx, dr, dw, ws)
        ds, err, dw64, dw_err = bwd_reference(dy, dres if with_dres else None, s, w, rstd)
        for got in (dx, dr):
            h = half_step(got.dtype)
            assert ((got.cpu().double() - ds).abs() <= err * (1 + h) + h * ds.abs()).all()
        assert ((dw.cpu().double() - dw64).abs() <= dw_err + 1e-30).all()
        # the gradient's outputs one by one, and dres over dres_out
        dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
        rom.rom_add_rmsnorm_bwd(d[0], d[1] if with_dres else None, d[2], d[3], d[4], dx2, None, None, None)
        rom.rom_add_rmsnorm_bwd(d[0], d[1] if with_dres else None, d[2], d[3], d[4], None, None, dw2, ws)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        if with_dres:
            over = d[1].clone()
            rom.rom_add_rmsnorm_bwd(d[0], over, d[2], d[3], d[4], None, over, None, None)
            assert torch.equal(over, dr)


@gpu
def test_add_rmsnorm_gradient_matches_differences():
    """Central differences of <y, dy> + <res_out, dres> of the float32 kernel,
    along random directions of x and w. The forward's float32 error over the
    step (1e-2) bounds the rounding part; the step's own part is third order:
    both measured in 64 bits by the formula beside it."""
    T, D, eps, h = 5, 264, 1e-5, 1e-2
    x, res, w = make_rows(T, D, F32, F32, seed=3)
    g = torch.Generator().manual_seed(4)
    dy, dres, vx = (torch.randn(T, D, generator=g) for _ in range(3))
    vw = torch.randn(D, generator=g)

    def loss(x_, w_):
        o = run_norm(x_, res, w_, eps, F32, q8=False)
        return (o["y"].double() * dy.double()).sum() + (o["res_out"].double() * dres.double()).sum()

    def loss64(x_, w_):
        s = x_.double() + res.double()
        y = s * (s.square().mean(-1, keepdim=True) + eps).rsqrt() * w_.double()
        return (y * dy.double()).sum() + (s * dres.double()).sum()

    n = rom.add_rmsnorm(x.cuda(), res.cuda(), w.cuda(), eps)
    gr = rom.add_rmsnorm_backward(dy.cuda(), n, w.cuda(), dres.cuda())
    for dx_, dw_, along in ((vx, 0 * vw, (gr.dx.cpu().double() * vx.double()).sum()),
                            (0 * vx, vw, (gr.dw.cpu().double() * vw.double()).sum())):
        hi, lo = (x + h * dx_, w + h * dw_), (x - h * dx_, w - h * dw_)
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        exact = (loss64(*hi) - loss64(*lo)) / (2 * h)
        # rounding of each output: 40 U of it (the forward's bound), twice, over 2 h
        s = (x + res).double().abs()
        y = s * n.rstd.cpu().double()[:, None] * w.double().abs()
        noise = 2 * 40 * U * ((y + 1) * dy.double().abs() + (s + 1) * dres.double().abs()).sum() / (2 * h)
        assert abs(num - exact) <= noise
        # the formula's own difference quotient: third order in h
        third = abs((loss64(x + 2 * h * dx_, w + 2 * h * dw_) - loss64(x - 2 * h * dx_, w - 2 * h * dw_)) / (4 * h) - exact)
        assert abs(along - num) <= third + 2 * noise


@gpu
def test_add_rmsnorm_repeats_bit_for_bit_and_empty_batches():
    dy, dres, w = make_rows(2000, 264, BF16, F32, seed=9)
    _, s, _ = make_rows(2000, 264, BF16, F32, seed=10)
    rstd = (s.double().square().mean(-1) + 1e-5).rsqrt().float()
    d = [t.cuda() for t in (dy, dres, s, w, rstd)]
    got = []
    for _ in range(3):
        dw = torch.empty(264, device="cuda")
        ws = torch.empty(rom.rom_add_rmsnorm_bwd_workspace_size(2000, 264), dtype=torch.uint8, device="cuda")
        rom.rom_add_rmsnorm_bwd(*d, None, None, dw, ws)
        got.append(dw.cpu())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    e = rom.add_rmsnorm(torch.empty(0, 64, dtype=BF16, device="cuda"), None, torch.ones(64, device="cuda"), q8=True)
    assert e.y.shape == (0, 64)
    gr = rom.add_rmsnorm_backward(torch.empty(0, 64, dtype=BF16, device="cuda"), e, torch.ones(64, device="cuda"))
    assert (gr.dw.cpu() == 0).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,K", [(1, 8), (69, 64), (131, 104), (77, 264), (9, 1000), (5, 4096), (3, 16384)])
def test_quant_rows_gives_the_definitions_codes(rows, K, dtype):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(rows, K, generator=g) * 10.0 ** torch.randint(-20, 20, (rows, 1), generator=g)).to(dtype)
    x[0] = 0
    if rows > 3:
        x[1, 3] = float("nan")
        x[2, K - 1] = -float("inf")
    q, s = rom.quant_rows(x.cuda())
    rq, rs = rows_to_8bit(x)
    q, s = q.cpu(), s.cpu()
    for r in range(rows):
        if not x[r].float().isfinite().all():
            assert s[r].isnan() and q[r].float().isnan().all()
        else:
            assert torch.equal(q[r].view(torch.uint8), rq[r].view(torch.uint8)) and s[r] == rs[r], r


@gpu
def test_norm_on_another_stream_and_in_a_graph():
    x, res, w = (t.cuda() for t in make_rows(40, 1000, BF16, F32, seed=5))
    ref = rom.add_rmsnorm(x, res, w, q8=True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = rom.add_rmsnorm(x, res, w, q8=True, stream=st)
    grads = rom.add_rmsnorm_backward(other.y, other, w, stream=st)
    st.synchronize()
    assert torch.equal(other.y, ref.y) and torch.equal(other.residual, ref.residual)
    bufs = rom.NormBuffers(40, 1000, BF16, F32, "cuda", q8=True)
    gb = rom.NormGrads(40, 1000, BF16, F32, "cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rom.add_rmsnorm(x, res, w, q8=True, bufs=bufs)
        rom.add_rmsnorm_backward(bufs.y, bufs, w, bufs=gb)
    for _ in range(2):
        bufs.y.zero_()
        gb.dw.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.y, ref.y) and torch.equal(bufs.y8.view(torch.uint8), ref.y8.view(torch.uint8))
        assert torch.equal(gb.dw, grads.dw) and torch.equal(gb.dx, grads.dx)


@gpu
def test_binding_refuses_wrong_tensors():
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    y, res = torch.empty_like(x), torch.zeros(4, 64, device="cuda")
    for bad, match in ((dict(weight=w.to(BF16)), "weight must be"), (dict(weight=w[:32]), "weight must be"),
                       (dict(y=y[:3]), "y must be"), (dict(y=res), "y must be"),
                       (dict(res_out=y), "res_out must be"), (dict(residual=res.t()), "residual must be"),
                       (dict(rstd=torch.empty(5, device="cuda")), "rstd must be"),
                       (dict(weight=w.cpu()), "contiguous CUDA"), (dict(y8=torch.empty(4, 64, dtype=E4M3, device="cuda")), "INVALID"),
                       (dict(x=torch.zeros(64, 4, dtype=BF16, device="cuda").t()), "contiguous CUDA")):
        a = dict(x=x, residual=res, weight=w, eps=1e-5, res_out=res, y=y)
        a.update(bad)
        with pytest.raises(rom.RomError, match=match):
            rom.rom_add_rmsnorm(**a)
    with pytest.raises(rom.RomError, match="q must be"):
        rom.rom_quant_rows(x, torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, device="cuda"))
    with pytest.raises(rom.RomError, match="WORKSPACE"):
        rom.rom_add_rmsnorm_bwd(x, None, res, w, torch.ones(4, device="cuda"), y, None, w.clone(), None)


@gpu
def test_rows_past_two_to_the_31_elements():
    """A batch of more than 2^31 elements: its last rows are those of a small
    batch (a row's result does not depend on the others)."""
    D = 8192
    T = (1 << 31) // D + 3
    x = torch.empty(T, D, dtype=BF16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    w = torch.ones(D, device="cuda")
    n = rom.add_rmsnorm(x, None, w, q8=True, residual_dtype=BF16)
    m = rom.add_rmsnorm(x[-4:].contiguous(), None, w, q8=True, residual_dtype=BF16)
    for a, b in ((n.y, m.y), (n.residual, m.residual), (n.y8.view(torch.uint8), m.y8.view(torch.uint8)),
                 (n.y_scale, m.y_scale), (n.rstd, m.rstd)):
        assert torch.equal(a[-4:], b)
    q, s = rom.quant_rows(n.y)
    q4, s4 = rom.quant_rows(m.y)
    assert torch.equal(q[-4:].view(torch.uint8), q4.view(torch.uint8)) and torch.equal(s[-4:], s4)
    del n.y8, q
    dx = torch.empty_like(x)
    rom.rom_add_rmsnorm_bwd(n.y, None, n.residual, w, n.rstd, dx, None, None, None)
    dx4 = torch.empty_like(m.y)
    rom.rom_add_rmsnorm_bwd(m.y, None, m.residual, w, m.rstd, dx4, None, None, None)
    assert torch.equal(dx[-4:], dx4)
