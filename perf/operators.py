"""Measured cases of three operators that stand around the expert projections.

* ``norm`` / ``norm_bwd``: the addition of the residual and the root-mean-square
  norm in front of a block (rom_add_rmsnorm), its rows written in the
  activations' type and in 8 bits (e4m3) with a scale per row, and its gradient.
* ``q8``: the block's products grouped by expert (Conv+Gate, Out) on rows and
  weights in 8 bits (rom_expert_proj_q8).
* ``w4``: the routed projection of up to 64 tokens on weights in 4 bits with a
  scale per group (rom_expert_proj_w4).

``run`` computes them in their plain form (elementary torch operations in
float32), or, where ``own`` is true, calls the library.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100


def listed():
    return [
        # One decoded token of the Swimba in-projection's width: latency.
        dict(name="norm_decode_1x4096", op="norm", T=1, D=4096, dtype="bf16", res="f32", q8=True, eps=1e-5),
        # The norm in front of the prefill batch, float32 residual stream, 8-bit rows for the experts.
        dict(name="norm_prefill_16384x2048", op="norm", T=16384, D=2048, dtype="bf16", res="f32", q8=True, eps=1e-5),
        # A ragged batch of a width that is no multiple of a warp, float32 throughout.
        dict(name="norm_ragged_1237x1000_f32", op="norm", T=1237, D=1000, dtype="f32", res="f32", q8=False, eps=1e-6),
        # The gradient in the top-2 training step, residual stream in bf16.
        dict(name="norm_bwd_32768x2560", op="norm_bwd", T=32768, D=2560, dtype="bf16", res="bf16", q8=False, eps=1e-5),
        # A short sequence's gradient, float32 residual stream.
        dict(name="norm_bwd_517x1024", op="norm_bwd", T=517, D=1024, dtype="bf16", res="f32", q8=False, eps=1e-5),
        # The prefill block's Conv+Gate products (16384 tokens, d_model 2048, d_inner 4096, 8 experts).
        dict(name="q8_conv_gate_prefill", op="q8", proj="conv_gate", T=16384, K=2048, N=4096, E=8, k=1, skew=0.0),
        # Its Out products.
        dict(name="q8_out_prefill", op="q8", proj="out", T=16384, K=4096, N=2048, E=8, k=1, skew=0.0),
        # Top-2 Out of an uneven batch over 16 experts, some of them with few rows or none.
        dict(name="q8_out_uneven_top2", op="q8", proj="out", T=1537, K=2048, N=1024, E=16, k=2, skew=2.0),
        # A decode batch's Out products: the weights' bytes count.
        dict(name="q8_out_decode_64", op="q8", proj="out", T=64, K=4096, N=2048, E=8, k=1, skew=0.0),
        # One token through the Swimba in-projection (X | B | C columns, 4 experts).
        dict(name="w4_inproj_1", op="w4", proj="inproj", T=1, K=4096, N=10240, E=4, k=1, group=128),
        # A decode batch of 64 through the same projection.
        dict(name="w4_inproj_64", op="w4", proj="inproj", T=64, K=4096, N=10240, E=4, k=1, group=128),
        # Top-2 Conv and Gate of a small batch, 16 experts, fine groups, sizes that fill no tile.
        dict(name="w4_conv_gate_19_top2", op="w4", proj="conv_gate", T=19, K=1000, N=2004, E=16, k=2, group=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "q8", "w4"])
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        D = 8 * _log_int(rng, 8, 1024)
        T = _log_int(rng, 1, min(32768, 32768 * 2560 // D))
        return dict(op=op, T=T, D=D, dtype=dtype, res=rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32",
                    q8=op == "norm" and rng.random() < 0.6, eps=rng.choice([1e-5, 1e-6]))
    if op == "q8":
        proj = rng.choice(["conv_gate", "out"])
        k = 1 if proj == "conv_gate" else rng.choice([1, 1, 2])
        E = rng.choice([2, 4, 8, 16, 33, 64])
        K, N = 16 * _log_int(rng, 8, 320), 128 * _log_int(rng, 1, 40)
        most = 2 * 16384 * 2048 * 4096 // (k * K * N * (2 if proj == "conv_gate" else 1))
        return dict(op=op, proj=proj, T=_log_int(rng, 1, max(1, min(16384, most))), K=K, N=N, E=E, k=k,
                    skew=rng.choice([0.0, 0.5, 2.0]))
    proj = rng.choice(["inproj", "inproj", "conv_gate"])
    E = rng.choice([1, 4, 8, 16])
    K = 8 * _log_int(rng, 8, 640)
    m = 2 if proj == "conv_gate" else 1
    N = _log_int(rng, 8, max(8, min(10240, 4 * 10240 * 4096 // (E * K * m))))
    return dict(op=op, proj=proj, T=_log_int(rng, 1, 64), K=K, N=N, E=E, k=min(E, rng.choice([1, 1, 2, 3])),
                group=rng.choice([32, 64, 128]))


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows_to_8bit(v):
    """Rows of v in e4m3 with a scale per row (float32)."""
    scale = v.abs().amax(-1).clamp(min=SCALE_FLOOR) / E4M3_MAX
    return (v / scale.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _routing(gen, T, E, k, skew):
    """A routing of T tokens: experts of every slot, weights, and the expert order of the slots."""
    bias = -skew * torch.arange(E, device="cuda", dtype=torch.float32) / max(1, E - 1) * 3.0
    logits = torch.randn((T, E), generator=gen, device="cuda") + bias
    top, idx = logits.topk(k, dim=-1)
    idx = idx.to(torch.int32).contiguous()
    order = torch.argsort(idx.flatten().to(torch.int64), stable=True).to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(idx.flatten().to(torch.int64), minlength=E).cumsum(0).to(torch.int32)
    return idx, top.softmax(-1).contiguous(), order.contiguous(), offsets


def _weights_to_4bit(w, group):
    """w [E, N, K] float32 -> the library's 4-bit storage: q uint8 [E, N16, K128, 2, 8, 4, 16]
    (tiles of 16 rows x 128 columns, 1 KB each) and scales bf16 [E, N16, K128, 16, 128 / group]."""
    E, N, K = w.shape
    nt, kb = -(-N // 16), -(-K // 128)
    w = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nt * 16 - N))
    g = w.view(E, nt, 16, kb, 128 // group, group)
    s = (g.abs().amax(-1) / 7.0).to(torch.bfloat16)
    sf = s.float().unsqueeze(-1)
    q = torch.where(sf > 0, torch.round(g / sf), torch.zeros_like(g)).clamp(-8, 7).to(torch.int32) + 8
    # row = (n16, half, 8 rows); column = (k128, word, step parity, quad lane, element)
    q = q.view(E, nt, 2, 8, kb, 4, 2, 4, 2, 2)  # .., word, p1, lane, p0, p2
    q = q.permute(0, 1, 4, 2, 3, 7, 5, 9, 6, 8)  # E, n16, k128, half, row, lane, word, p2, p1, p0
    q = q.reshape(E, nt, kb, 2, 8, 4, 16, 2)     # nibbles of a byte: low first
    q = (q[..., 0] | (q[..., 1] << 4)).to(torch.uint8).contiguous()
    return q, s.permute(0, 1, 3, 2, 4).contiguous()


def _weights_from_4bit(q, s, N, K):
    """The float32 values [E, N, K] that the 4-bit storage stands for."""
    E, nt, kb = q.shape[:3]
    group = 128 // s.shape[-1]
    v = torch.stack((q & 15, q >> 4), -1).to(torch.float32) - 8.0
    v = v.view(E, nt, kb, 2, 8, 4, 4, 2, 2, 2).permute(0, 1, 3, 4, 2, 6, 8, 5, 9, 7)
    v = v.reshape(E, nt * 16, kb, 128 // group, group)
    sf = s.permute(0, 1, 3, 2, 4).reshape(E, nt * 16, kb, 128 // group, 1).float()
    return (v * sf).view(E, nt * 16, kb * 128)[:, :N, :K]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        T, D, dt, rt = case["T"], case["D"], _dt(case["dtype"]), _dt(case["res"])
        s["w"] = 1.0 + 0.1 * normal(D)
        if op == "norm":
            s["x"] = normal(T, D).to(dt)
            # the residual stream grows over the layers and is uneven over the channels
            s["residual"] = (normal(T, D) * (1.0 + 2.0 * normal(D).abs())).to(rt)
            s["res_out"], s["y"] = torch.empty((T, D), dtype=rt, device="cuda"), torch.empty((T, D), dtype=dt, device="cuda")
            s["rstd"] = torch.empty(T, device="cuda")
            s["y8"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device="cuda") if case["q8"] else None
            s["y_scale"] = torch.empty(T, device="cuda") if case["q8"] else None
        else:
            s["dy"], s["dres_out"] = normal(T, D).to(dt), normal(T, D).to(rt)
            s["res_out"] = (normal(T, D) * (1.0 + 2.0 * normal(D).abs())).to(rt)
            s["rstd"] = torch.rsqrt(s["res_out"].double().square().mean(-1) + case["eps"]).float()
            s["dx"] = torch.empty((T, D), dtype=dt, device="cuda")
            s["dres"] = torch.empty((T, D), dtype=rt, device="cuda")
            s["dw"] = torch.empty(D, device="cuda")
            s["ws"] = torch.empty(min(T, 512) * D, device="cuda")  # the call's workspace
        return s
    T, K, N, E, k = case["T"], case["K"], case["N"], case["E"], case["k"]
    if op == "q8":
        s["topk_idx"], s["topk_w"], s["sorted_slot"], s["offsets"] = _routing(gen, T, E, k, case["skew"])
        gate = case["proj"] == "conv_gate"
        # rows in expert order: normed activations for Conv+Gate, gated products for Out
        rows = normal(T, K) if gate else normal(T, K) * torch.nn.functional.silu(normal(T, K))
        s["a"], s["a_scale"] = _rows_to_8bit(rows[(s["sorted_slot"] // k).long()])
        for i in range(2 if gate else 1):
            s["w%d" % i], s["w%d_scale" % i] = _rows_to_8bit(normal(E, N, K) / math.sqrt(K))
        s["slots"] = torch.empty((T * k, N), device="cuda") if k > 1 else None
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        return s
    s["topk_idx"], s["topk_w"], _, _ = _routing(gen, T, E, k, 0.0)
    s["x"] = normal(T, K).to(torch.bfloat16)
    m = 2 if case["proj"] == "conv_gate" else 1
    for i in range(m):
        s["q%d" % i], s["s%d" % i] = _weights_to_4bit(normal(E, N, K) / math.sqrt(K), case["group"])
    if m == 2:
        s["out"] = torch.empty((2, T * k, N), device="cuda")
    elif k > 1:
        s["out"] = torch.empty((T * k, N), device="cuda")
    else:
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from mixture_experts_projections_b200 import rom
    op = s["op"]
    if op == "norm":
        rom.rom_add_rmsnorm(s["x"], s["residual"], s["w"], s["eps"], s["res_out"], s["y"], s["y8"], s["y_scale"], s["rstd"])
        return {n: s[n] for n in ("res_out", "y", "y8", "y_scale", "rstd")}
    if op == "norm_bwd":
        rom.rom_add_rmsnorm_bwd(s["dy"], s["dres_out"], s["res_out"], s["w"], s["rstd"], s["dx"], s["dres"], s["dw"], s["ws"])
        return {n: s[n] for n in ("dx", "dres", "dw")}
    if op == "q8":
        gate = s["proj"] == "conv_gate"
        rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE if gate else rom.ROM_PROJ_OUT, s["a"], s["a_scale"], s["w0"],
                               s["w0_scale"], s.get("w1"), s.get("w1_scale"), s["k"], s["offsets"], s["sorted_slot"],
                               s["topk_w"], s["out"] if s["k"] == 1 else s["slots"])
        if s["k"] > 1:
            rom.rom_combine(rom.ROM_COMBINE_SUM, rom.ROM_BF16, s["slots"], s["T"], s["k"], s["N"], None, s["out"])
        return s["out"]
    gate = s["proj"] == "conv_gate"
    rom.rom_expert_proj_w4(rom.ROM_PROJ_CONV_GATE_SLOTS if gate else rom.ROM_PROJ_INPROJ, s["x"], s["q0"], s["s0"],
                           s.get("q1"), s.get("s1"), s["N"], s["k"], s["topk_idx"], s["topk_w"], s["out"])
    return s["out"]


def _plain(s):
    op = s["op"]
    if op == "norm":
        dt = s["x"].dtype
        res = (s["residual"].float() + s["x"].float()).to(s["residual"].dtype)
        r = res.float()
        rstd = torch.rsqrt(r.square().mean(-1) + s["eps"])
        y = r * rstd.unsqueeze(-1) * s["w"]
        y8, scale = _rows_to_8bit(y) if s["q8"] else (None, None)
        return {"res_out": res, "y": y.to(dt), "y8": y8, "y_scale": scale, "rstd": rstd}
    if op == "norm_bwd":
        r, dy, rstd = s["res_out"].float(), s["dy"].float(), s["rstd"].unsqueeze(-1)
        g = dy * s["w"]
        ds = s["dres_out"].float() + rstd * (g - r * rstd.square() * (g * r).mean(-1, keepdim=True))
        return {"dx": ds.to(s["dy"].dtype), "dres": ds.to(s["res_out"].dtype), "dw": (dy * r * rstd).sum(0)}
    T, N, k = s["T"], s["N"], s["k"]
    if op == "q8":
        off = s["offsets"].tolist()
        outs = []
        for w, scale in ((s["w0"], s["w0_scale"]), (s.get("w1"), s.get("w1_scale"))):
            if w is not None:
                # one product per expert over its own rows
                v = torch.cat([s["a"][a:b].float() @ w[e].float().t() * scale[e] for e, (a, b) in enumerate(zip(off, off[1:]))])
                outs.append(v * s["a_scale"].unsqueeze(-1))
        if len(outs) == 2:
            return (outs[0] * (outs[1] * torch.sigmoid(outs[1]))).to(torch.bfloat16)
        slot = s["sorted_slot"].long()
        v = torch.empty_like(outs[0])
        v[slot] = outs[0] * s["topk_w"].flatten()[slot].unsqueeze(-1)
        return v.view(T, k, N).sum(1).to(torch.bfloat16)
    x, idx = s["x"].float(), s["topk_idx"].long()
    tok = torch.arange(T, device="cuda").unsqueeze(-1)
    outs = []
    for q, scale in ((s["q0"], s["s0"]), (s.get("q1"), s.get("s1"))):
        if q is not None:
            # every expert's product with every token, then each slot's own
            every = torch.matmul(x, _weights_from_4bit(q, scale, N, s["K"]).transpose(1, 2))
            outs.append(every[idx, tok].reshape(T * k, N))
    if len(outs) == 2:
        return torch.stack(outs)
    v = outs[0] * s["topk_w"].flatten().unsqueeze(-1)
    return v.to(torch.bfloat16) if k == 1 else v


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, T, D = case["T"] * case["D"], case["T"], case["D"]
        a, r = (2 if case["dtype"] == "bf16" else 4), (2 if case["res"] == "bf16" else 4)
        if op == "norm":
            return {"bytes": n * (2 * a + 2 * r + (1 if case["q8"] else 0)) + 4 * D + T * (8 if case["q8"] else 4),
                    "flops": n * (8 if case["q8"] else 6)}
        return {"bytes": n * (2 * a + 3 * r) + 8 * D + 4 * T, "flops": 12 * n}
    T, K, N, E, k = case["T"], case["K"], case["N"], case["E"], case["k"]
    m = 2 if case["proj"] == "conv_gate" else 1
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that have rows, of an even routing
    if op == "q8":
        return {"bytes": T * k * (K + 12) + used * m * N * (K + 4) + 2 * T * N, "flops": 2 * m * T * k * K * N}
    wide = 4 * m * k if (m == 2 or k > 1) else 2
    return {"bytes": used * m * N * (K / 2 + 2 * K / case["group"]) + 2 * T * K + 8 * T * k + wide * T * N,
            "flops": 2 * m * T * k * K * N}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # the norm is that of the residual as it is stored
        total = s["x"].double() + s["residual"].double()
        r = total.to(s["residual"].dtype).double()
        rstd = (r.pow(2).sum(-1) / case["D"] + case["eps"]).pow(-0.5)
        y = torch.einsum("td,t,d->td", r, rstd, s["w"].double())
        scale = torch.maximum(y.amax(-1), (-y).amax(-1)).clamp(min=SCALE_FLOOR) / E4M3_MAX
        q8 = case["q8"]
        return {"res_out": total, "y": y, "y8": y / scale[:, None] if q8 else None, "y_scale": scale if q8 else None, "rstd": rstd}
    if op == "norm_bwd":
        r, dy, w, i = s["res_out"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
        n = r * i[:, None]
        along = torch.einsum("td,td,d->t", n, dy, w) / case["D"]
        ds = s["dres_out"].double() + i[:, None] * (dy * w - n * along[:, None])
        return {"dx": ds, "dres": ds, "dw": torch.einsum("td,td->d", n, dy)}
    k, N, E, T = case["k"], case["N"], case["E"], case["T"]
    if op == "q8":
        slot = s["sorted_slot"].long()
        expert = s["topk_idx"].flatten().long()[slot]
        a = s["a"].double() * s["a_scale"].double()[:, None]
        out = []
        for i in range(2 if case["proj"] == "conv_gate" else 1):
            v = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
            for e in range(E):
                mine = (expert == e).nonzero().flatten()
                v[mine] = a[mine] @ (s["w%d" % i][e].double() * s["w%d_scale" % i][e].double()[:, None]).t()
            out.append(v)
        if len(out) == 2:
            return out[0] * out[1] / (1.0 + torch.exp(-out[1]))
        total = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        return total.index_add_(0, slot // k, out[0] * s["topk_w"].double().flatten()[slot, None])
    x = s["x"].double()
    out = []
    for i in range(2 if case["proj"] == "conv_gate" else 1):
        w = _weights_from_4bit(s["q%d" % i], s["s%d" % i], N, case["K"])
        v = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
        for e in range(E):
            t, j = (s["topk_idx"] == e).nonzero(as_tuple=True)
            v[t * k + j] = x[t] @ w[e].double().t()
        out.append(v)
    if len(out) == 2:
        return torch.stack(out)
    return out[0] * s["topk_w"].double().reshape(-1, 1)
