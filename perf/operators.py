"""The operators around the MoE layer, as measured cases.

Five operators: the norm before a block (``norm_in``), the norm after it with
its gate and residual scale (``norm_out``, optionally with the next block's
norm), the AdamW step over many tensors (``adamw``), the dense product of e4m3
codes with a scale per block of 128 (``matmul``) and the grouped SwiGLU experts
on such codes (``experts``).
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
E5M2_MAX = 57344.0
STATE_BLOCK = 256


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # the norm before a layer of hidden size 4096, for a ragged batch of prompts
        dict(name="norm_in fwd 333", kind="norm_in", dir="fwd", T=333, H=4096, x="bf16", w="fp32", res=False),
        # its backward in training at hidden size 2048, with an fp32 residual stream
        dict(name="norm_in bwd 4096", kind="norm_in", dir="bwd", T=4096, H=2048, x="fp32", w="fp32", res=True),
        # one decoded token: the norm after a block and the next block's norm
        dict(name="norm_out fwd 1", kind="norm_out", dir="fwd", T=1, H=2048, x="bf16", w="bf16", gate="token", next=True),
        # the same for a training batch
        dict(name="norm_out fwd 16k", kind="norm_out", dir="fwd", T=16384, H=2048, x="bf16", w="fp32", gate="token",
             next=True),
        # its backward at hidden size 4096
        dict(name="norm_out bwd 16k", kind="norm_out", dir="bwd", T=16384, H=4096, x="bf16", w="fp32", gate="token",
             next=True),
        # a block's small parameters: router, norms, biases, many of odd sizes
        dict(name="adamw32 small", kind="adamw", bits=32, sizes="262144,2048,2048,8,128,4095,1,777,65537,2048,33,100001",
             p="bf16", g="bf16", master=True),
        # the experts of a layer with E=128, H=2048, I=768: bf16 weights, fp32 masters and gradients
        dict(name="adamw32 layer", kind="adamw", bits=32, sizes="402653184,201326592,262144,2048,2048", p="bf16",
             g="fp32", master=True),
        # 16 experts of H=4096, I=1536 with 8-bit states
        dict(name="adamw8 layer", kind="adamw", bits=8, sizes="201326592,100663296,65536,4096,4096", p="bf16", g="fp32",
             master=True),
        # a projection of a few decoded tokens
        dict(name="matmul decode 7", kind="matmul", M=7, N=4096, K=2048),
        # a projection of a ragged prompt batch
        dict(name="matmul 4097", kind="matmul", M=4097, N=4096, K=4096),
        # one decoded token through its 8 of 128 experts
        dict(name="experts decode 1", kind="experts", T=1, H=2048, E=128, K=8, I=768),
        # a prompt batch through them
        dict(name="experts 4096", kind="experts", T=4096, H=2048, E=128, K=8, I=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_in", "norm_out", "adamw", "matmul", "experts"])
    if kind in ("norm_in", "norm_out"):
        H = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            H = max(8, H // 8 * 8)      # most models; the others are odd
        T = max(1, min(_log(rng, 1, 16384), 16384 * 4096 // H))
        c = dict(kind=kind, dir=rng.choice(["fwd", "bwd"]), T=T, H=H, x=rng.choice(["bf16", "fp32"]),
                 w=rng.choice(["bf16", "fp32"]))
        if kind == "norm_in":
            c["res"] = c["dir"] == "bwd" and rng.random() < 0.7
        else:
            c.update(gate=rng.choice(["none", "token", "element"]), next=rng.random() < 0.6)
        return c
    if kind == "adamw":
        total, count = _log(rng, 3000, 150_000_000), rng.randint(1, 10)
        cuts = [rng.random() ** 3 + 1e-3 for _ in range(count)]
        sizes = [max(1, int(total * c / sum(cuts))) for c in cuts]
        p = rng.choice(["bf16", "fp32"])
        return dict(kind=kind, bits=rng.choice([32, 8]), sizes=",".join(map(str, sizes)), p=p,
                    g=rng.choice(["bf16", "fp32"]), master=p == "bf16" and rng.random() < 0.7)
    if kind == "matmul":
        N, K = _log(rng, 64, 8192), max(16, _log(rng, 128, 8192) // 16 * 16)
        M = max(1, min(_log(rng, 1, 8192), 4097 * 4096 * 4096 // (N * K)))
        return dict(kind=kind, M=M, N=N, K=K)
    E = rng.choice([8, 16, 32, 64, 128])
    K = rng.choice([1, 2, 4, 8])
    H, I = 256 * rng.randint(1, 11 if E < 128 else 8), 128 * rng.randint(1, 8 if E < 128 else 6)
    return dict(kind=kind, T=_log(rng, 1, 4096), H=H, E=E, K=K, I=I)


# ---------------------------------------------------------------- the inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS, LR, B1, B2, ADAM_EPS, WD, STEP, SEED, RES_SCALE = 1e-6, 3e-4, 0.9, 0.95, 1e-8, 0.1, 100, 1234, 0.75


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    return {"norm_in": _prepare_norm, "norm_out": _prepare_norm, "adamw": _prepare_adamw,
            "matmul": _prepare_matmul, "experts": _prepare_experts}[case["kind"]](case, g)


def _prepare_norm(c, g):
    T, H, xt, wt = c["T"], c["H"], _TYPES[c["x"]], _TYPES[c["w"]]
    s = dict(case=c, x=_randn(g, T, H, dtype=xt, std=2.0), w=_randn(g, H, dtype=wt, std=0.1, mean=1.0))
    if c["kind"] == "norm_in":
        if c["dir"] == "bwd":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["grad_n"] = _randn(g, T, H, dtype=torch.bfloat16)
            s["grad_res"] = _randn(g, T, H, dtype=xt) if c["res"] else None
        return s
    s["y"] = _randn(g, T, H, dtype=torch.bfloat16)
    s["gate"] = {"none": lambda: None, "token": lambda: _randn(g, T),
                 "element": lambda: _randn(g, T, H, dtype=torch.bfloat16)}[c["gate"]]()
    s["w2"] = _randn(g, H, dtype=wt, std=0.1, mean=1.0) if c["next"] else None
    if c["dir"] == "bwd":
        s["rstd"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS)
        s["out"] = s.pop("x")           # the forward's result, kept for its backward
        s["rstd2"] = torch.rsqrt(s["out"].float().square().mean(1) + EPS) if c["next"] else None
        s["grad_out"] = _randn(g, T, H, dtype=xt)
        s["grad_next"] = _randn(g, T, H, dtype=torch.bfloat16) if c["next"] else None
    return s


def _prepare_adamw(c, g):
    s = dict(case=c, step=STEP, params=[], grads=[], master=[], m=[], v=[], m_scale=[], v_scale=[])
    for n in map(int, c["sizes"].split(",")):
        w = _randn(g, n, std=0.02)
        s["params"].append(w.to(_TYPES[c["p"]]))
        s["master"].append(w if c["master"] else None)
        s["grads"].append(_randn(g, n, dtype=_TYPES[c["g"]], std=1e-3))
        # the averages of earlier steps' gradients, with the spread they have in training
        m = _randn(g, n, std=3e-4)
        v = (torch.randn(n, generator=g, device=DEV) * 1.5 - 14).exp_()
        if c["bits"] == 8:
            m, ms = _blocks(m, E4M3_MAX)
            v, vs = _blocks(v, E5M2_MAX)
            m = m.to(torch.float8_e4m3fn).view(torch.uint8)[:n].clone()
            v = v.to(torch.float8_e5m2).view(torch.uint8)[:n].clone()
            s["m_scale"].append(ms)
            s["v_scale"].append(vs)
        s["m"].append(m)
        s["v"].append(v)
        del w, m, v
    if own:  # the optimiser object that a training program keeps
        import combine_topk_multihot_gb300 as moe
        s["opt"] = moe.AdamWState(s["params"], state_bits=c["bits"], master=s["master"] if c["master"] else None,
                                  seed=SEED, step=STEP, exp_avg=s["m"], exp_avg_sq=s["v"],
                                  exp_avg_scale=s["m_scale"] or None, exp_avg_sq_scale=s["v_scale"] or None)
    return s


def _blocks(v, top):
    """(values over their block's scale, scales) of a flat tensor, padded to whole blocks."""
    b = torch.nn.functional.pad(v, (0, -v.numel() % STATE_BLOCK)).view(-1, STATE_BLOCK)
    amax = b.abs().amax(1)
    scale = (amax / torch.full_like(amax, top)).clamp_min(2.0 ** -120)   # a tensor's division is not a product
    return (b * (1.0 / scale)[:, None]).view(-1), scale


def _quantize(v, block_rows):
    """e4m3 codes (as float8) of v [..., rows, cols] and a scale per block of block_rows x 128."""
    *lead, R, C = v.shape
    b = torch.nn.functional.pad(v.float(), (0, -C % 128, 0, -R % block_rows))
    nr, nc = b.shape[-2] // block_rows, b.shape[-1] // 128
    b = b.view(*lead, nr, block_rows, nc, 128)
    amax = b.abs().amax((-3, -1))
    scale = torch.where(amax > 0, (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(2.0 ** -126), torch.ones_like(amax))
    q = (b / scale[..., :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.view(*lead, nr * block_rows, nc * 128)[..., :R, :C].contiguous()
    return q.to(torch.float8_e4m3fn), scale


def _prepare_matmul(c, g):
    b, bs = _quantize(_randn(g, c["N"], c["K"], dtype=torch.bfloat16, std=0.02), 128)
    return dict(case=c, x=_randn(g, c["M"], c["K"], dtype=torch.bfloat16), b=b.view(torch.uint8), bs=bs)


def _prepare_experts(c, g):
    T, H, E, K, I = c["T"], c["H"], c["E"], c["K"], c["I"]
    idx = torch.randn(T, E, generator=g, device=DEV).topk(K, dim=1).indices
    p = torch.rand(T, K, generator=g, device=DEV) + 0.1
    p = p / p.sum(1, keepdim=True)
    # the rows of the expanded layout: grouped by expert, in token order within each group
    expert, order = idx.reshape(-1).sort(stable=True)
    token = order // K
    counts = torch.bincount(expert, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    R = T * K
    x = _randn(g, T, H, dtype=torch.bfloat16)
    token_row = torch.empty(R, dtype=torch.int64, device=DEV)
    token_row[order] = torch.arange(R, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(case=c, x_disp=x[token], expert=expert, offsets=offsets, place=torch.arange(R, device=DEV) - offsets[expert],
             most=int(counts.max()), weight=p.reshape(-1)[order].contiguous())
    s["layout"] = (counts.to(**i32), offsets.to(**i32), torch.tensor([R, R], **i32), token.to(**i32), expert.to(**i32),
                   s["weight"], token_row.view(T, K).sort(1).values.reshape(-1).to(**i32), torch.zeros(1, **i32))
    for name, shape in (("W1", (2 * I, H)), ("W2", (H, I))):
        q = torch.empty(E, *shape, dtype=torch.uint8, device=DEV)
        sc = torch.empty(E, -(-shape[0] // 128), -(-shape[1] // 128), device=DEV)
        for e in range(E):
            qe, sc[e] = _quantize(_randn(g, *shape, dtype=torch.bfloat16, std=0.02), 128)
            q[e] = qe.view(torch.uint8)
        s[name], s[name + "s"] = q, sc
    return s


# -------------------------------------------------------------------- a pass
def run(state):
    k = state["case"]["kind"]
    if own:
        import combine_topk_multihot_gb300 as moe
        return {"norm_in": _own_norm_in, "norm_out": _own_norm_out, "adamw": _own_adamw, "matmul": _own_matmul,
                "experts": _own_experts}[k](moe, state)
    return {"norm_in": _norm_in, "norm_out": _norm_out, "adamw": _adamw, "matmul": _matmul, "experts": _experts}[k](state)


def _own_norm_in(moe, s):
    if s["case"]["dir"] == "fwd":
        return moe.moe_norm_in(s["x"], s["w"], eps=EPS)[0]
    return moe.moe_norm_in_backward(s["grad_n"], s["x"], s["w"], s["rstd"], grad_res=s["grad_res"])


def _own_norm_out(moe, s):
    if s["case"]["dir"] == "fwd":
        out, _, nxt, _ = moe.moe_norm_out(s["x"], s["y"], s["w"], gate=s["gate"], residual_scale=RES_SCALE,
                                          next_weight=s["w2"], eps=EPS)
        return out, nxt
    return moe.moe_norm_out_backward(s["grad_out"], s["y"], s["w"], s["rstd"], gate=s["gate"], residual_scale=RES_SCALE,
                                     grad_next=s["grad_next"], out=s["out"] if s["case"]["next"] else None,
                                     next_weight=s["w2"], next_rstd=s["rstd2"])


def _own_adamw(moe, s):
    moe.moe_adamw_step(s["opt"], s["grads"], lr=LR, beta1=B1, beta2=B2, eps=ADAM_EPS, weight_decay=WD)
    return _adamw_outputs(s)


def _own_matmul(moe, s):
    a, a_scale = moe.moe_quantize_fp8_block(s["x"])
    out = moe.moe_matmul_fp8_block(a, a_scale, s["b"], s["bs"])
    return a.view(torch.float8_e4m3fn), a_scale, out


def _own_experts(moe, s):
    c = s["case"]
    layout = moe.Layout.from_tensors(c["T"], c["E"], c["K"], 1, s["layout"])
    return moe.moe_grouped_experts_fp8_block(s["x_disp"], layout, s["W1"], s["W1s"], s["W2"], s["W2s"])


def _norm_in(s):
    x, w = s["x"].float(), s["w"].float()
    if s["case"]["dir"] == "fwd":
        return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w).bfloat16()
    r, dn = s["rstd"][:, None], s["grad_n"].float()
    dx = r * (w * dn) - x * (r * r * r) * (w * dn * x).mean(1, keepdim=True)
    if s["grad_res"] is not None:
        dx = dx + s["grad_res"].float()
    return dx.to(s["x"].dtype), (dn * x * r).sum(0)


def _norm_out(s):
    c, y, w = s["case"], s["y"].float(), s["w"].float()
    gate = 1.0 if s["gate"] is None else torch.sigmoid(s["gate"].float())
    if c["gate"] == "token":
        gate = gate[:, None]
    if c["dir"] == "fwd":
        n = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * w
        out = (RES_SCALE * s["x"].float() + gate * n).to(s["x"].dtype)
        if not c["next"]:
            return out, None
        o = out.float()
        return out, (o * torch.rsqrt(o.square().mean(1, keepdim=True) + EPS) * s["w2"].float()).bfloat16()
    d, dw2, r = s["grad_out"].float(), None, s["rstd"][:, None]
    if c["next"]:
        o, dn2, r2 = s["out"].float(), s["grad_next"].float(), s["rstd2"][:, None]
        wd = s["w2"].float() * dn2
        d = d + r2 * wd - o * (r2 * r2 * r2) * (wd * o).mean(1, keepdim=True)
        dw2 = (dn2 * o * r2).sum(0)
    dgate = None
    if s["gate"] is not None:
        dgate = d * (y * r * w)
        if c["gate"] == "token":
            dgate = dgate.sum(1, keepdim=True)
        dgate = (gate * (1 - gate) * dgate).view(s["gate"].shape).to(s["gate"].dtype)
    dn = gate * d
    dy = r * (w * dn) - y * (r * r * r) * (w * dn * y).mean(1, keepdim=True)
    return (RES_SCALE * d).to(_TYPES[c["x"]]), dy.bfloat16(), dgate, (dn * y * r).sum(0), dw2


def _mix(x):
    """32 mixed bits of 32 bits, in int64 (the products' low halves)."""
    x = x ^ (x >> 16)
    x = (x * 0xA3D95B4F) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xC2F1E6D3) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random16(n, seed, tensor, step):
    """16 random bits for each of a tensor's n elements: two neighbours share a hash."""
    key = seed & 0xFFFFFFFF
    for k in (seed >> 32, tensor, step & 0xFFFFFFFF, step >> 32):
        key = _mix(key ^ k) + 0x9E3779B9 & 0xFFFFFFFF
    pair = torch.arange(-(-n // 2), device=DEV)
    h = _mix((pair & 0xFFFFFFFF) ^ _mix((pair >> 32) ^ key))
    return torch.stack([h & 0xFFFF, h >> 16], 1).view(-1)[:n]


def _adamw(s):
    """One step in 32 bits, each operation rounded once; the states and parameters in place."""
    c = s["case"]
    s["step"] += 1
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    lr_wd, step_size = f32(1.0 - LR * WD), f32(LR / (1 - B1 ** s["step"]))
    bc2 = f32(1.0 / math.sqrt(1 - B2 ** s["step"]))
    for i in range(len(s["params"])):
        p = s["master"][i] if c["master"] else s["params"][i].float()
        g, n = s["grads"][i].float(), p.numel()
        if c["bits"] == 8:
            m = _unblock(s["m"][i].view(torch.float8_e4m3fn), s["m_scale"][i])
            v = _unblock(s["v"][i].view(torch.float8_e5m2), s["v_scale"][i])
        else:
            m, v = s["m"][i], s["v"][i]
        m = m * f32(B1) + g * f32(1 - B1)
        v = v * f32(B2) + (g * g) * f32(1 - B2)
        p = p * lr_wd - step_size * (m / (v.sqrt() * bc2 + f32(ADAM_EPS)))
        if c["master"]:
            s["master"][i].copy_(p)
        s["params"][i].copy_(p)
        if c["bits"] == 8:
            q, ms = _blocks(m, E4M3_MAX)
            s["m"][i].copy_(q[:n].to(torch.float8_e4m3fn).view(torch.uint8))
            t, vs = _blocks(v, E5M2_MAX)
            # t's bits with its exponent moved to e5m2's place, 21 bits below a code's lowest; random ones added
            code = (t[:n] * 2.0 ** -112).view(torch.int32) + (_random16(n, SEED, i, s["step"]) << 5).int() >> 21
            s["v"][i].copy_(torch.where(v > 0, code.clamp(1, 0x7B), code))
            s["m_scale"][i].copy_(ms)
            s["v_scale"][i].copy_(vs)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
    return _adamw_outputs(s)


def _unblock(codes, scale):
    n = codes.numel()
    full = torch.nn.functional.pad(codes.float(), (0, -n % STATE_BLOCK)).view(-1, STATE_BLOCK)
    return (full * scale[:, None]).view(-1)[:n]


def _adamw_outputs(s):
    eight = s["case"]["bits"] == 8
    out = dict(params=s["params"], m=s["m"], v=s["v"])
    if s["case"]["master"]:
        out["master"] = s["master"]
    if eight:  # the codes as the numbers they stand for, in units of their block's scale
        out.update(m=[t.view(torch.float8_e4m3fn) for t in s["m"]], v=[t.view(torch.float8_e5m2) for t in s["v"]],
                   m_scale=s["m_scale"], v_scale=s["v_scale"])
    return out


def _expand(scale, block_rows, R, C):
    s = scale.repeat_interleave(128, -1)[..., :C]
    return s.repeat_interleave(block_rows, -2)[..., :R, :] if block_rows > 1 else s


def _matmul(s):
    a, sa = _quantize(s["x"], 1)
    b = s["b"].view(torch.float8_e4m3fn).float() * _expand(s["bs"], 128, *s["b"].shape)
    return a, sa, ((a.float() * _expand(sa, 1, *a.shape)) @ b.t()).bfloat16()


def _grouped(s, a, w, ws):
    """Each row times its expert's matrix: the rows in a block of equal height for each expert."""
    E, N, K = w.shape
    rows = a.new_zeros(E, s["most"], K)
    rows[s["expert"], s["place"]] = a
    full = w.view(torch.float8_e4m3fn).float() * _expand(ws, 128, N, K)
    return torch.bmm(rows, full.transpose(1, 2))[s["expert"], s["place"]]


def _experts(s):
    I = s["case"]["I"]
    a, sa = _quantize(s["x_disp"], 1)
    gu = _grouped(s, a.float() * _expand(sa, 1, *a.shape), s["W1"], s["W1s"])
    g, u = gu[:, :I], gu[:, I:]
    h, sh = _quantize(g / (1 + torch.exp(-g)) * u, 1)
    o = _grouped(s, h.float() * _expand(sh, 1, *h.shape), s["W2"], s["W2s"])
    return (o * s["weight"][:, None]).bfloat16()


# -------------------------------------------------------- the work of a pass
def work(case):
    c = case
    if c["kind"] in ("norm_in", "norm_out"):
        T, H, xb = c["T"], c["H"], 2 if c["x"] == "bf16" else 4
        if c["kind"] == "norm_in":
            row = xb + 2 if c["dir"] == "fwd" else 2 * xb + 2 + (xb if c["res"] else 0)
            return dict(bytes=T * H * row, flops=T * H * (4 if c["dir"] == "fwd" else 10))
        gate = {"none": 0, "token": 0, "element": 2}[c["gate"]]
        if c["dir"] == "fwd":
            return dict(bytes=T * H * (2 * xb + 2 + gate + (2 if c["next"] else 0)), flops=T * H * 10)
        return dict(bytes=T * H * (2 * xb + 4 + 2 * gate + (2 + xb if c["next"] else 0)), flops=T * H * 25)
    if c["kind"] == "adamw":
        n = sum(map(int, c["sizes"].split(",")))
        pb = 2 if c["p"] == "bf16" else 4
        one = (8 + pb if c["master"] else 2 * pb) + (2 if c["g"] == "bf16" else 4)
        return dict(bytes=n * (one + (16 if c["bits"] == 32 else 4 + 16 / STATE_BLOCK)), flops=n * 20)
    if c["kind"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(bytes=M * K * 2 + N * K + M * N * 2, flops=2 * M * N * K)
    R, H, I = c["T"] * c["K"], c["H"], c["I"]
    used = c["E"] * (1 - (1 - c["K"] / c["E"]) ** c["T"])     # experts that get a row
    return dict(bytes=int(used * 3 * H * I + R * H * 4), flops=6 * R * H * I)


# ---------------------------------------------- the same from 64-bit formulas
def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"norm_in": _exact_norm_in, "norm_out": _exact_norm_out, "adamw": _exact_adamw, "matmul": _exact_matmul,
            "experts": _exact_experts}[case["kind"]](case, f)


def _rms(v):
    return (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS).pow(-0.5)


def _exact_vjp(v, r, w, d):
    """Gradient of v r(v) w with respect to v, for the gradient d."""
    h = v * r
    t = d * w
    return r * (t - h * (t * h).sum(-1, keepdim=True) / v.shape[-1])


def _exact_norm_in(c, f):
    if c["dir"] == "fwd":
        return f["w"] * (f["x"] * _rms(f["x"]))
    r = f["rstd"].unsqueeze(-1)
    dx = _exact_vjp(f["x"], r, f["w"], f["grad_n"])
    if f["grad_res"] is not None:
        dx += f["grad_res"]
    return dx, torch.einsum("th,th,t->h", f["grad_n"], f["x"], f["rstd"])


def _exact_norm_out(c, f):
    T, H = f["y"].shape
    s = torch.ones(T, 1, dtype=torch.float64, device=DEV) if f["gate"] is None else 1 / (1 + torch.exp(-f["gate"]))
    s = s.reshape(T, -1)
    if c["dir"] == "fwd":
        out = RES_SCALE * f["x"] + s * (f["w"] * (f["y"] * _rms(f["y"])))
        if not c["next"]:
            return out, None
        held = out.to(_TYPES[c["x"]]).double()      # the next norm reads the stream as it is held
        return out, f["w2"] * (held * _rms(held))
    r = f["rstd"].unsqueeze(-1)
    hat = f["y"] * r
    d, dw2 = f["grad_out"], None
    if c["next"]:
        d = d + _exact_vjp(f["out"], f["rstd2"].unsqueeze(-1), f["w2"], f["grad_next"])
        dw2 = torch.einsum("th,th,t->h", f["grad_next"], f["out"], f["rstd2"])
    dgate = None
    if f["gate"] is not None:
        dgate = d * hat * f["w"] * s * (1 - s)
        dgate = dgate.sum(-1) if c["gate"] == "token" else dgate
    dn = d * s
    return RES_SCALE * d, _exact_vjp(f["y"], r, f["w"], dn), dgate, (dn * hat).sum(0), dw2


def _exact_adamw(c, s):
    t = STEP + 1
    out = dict(params=[], m=[], v=[])
    if c["master"]:
        out["master"] = []
    if c["bits"] == 8:
        out.update(m_scale=[], v_scale=[])
    for i, p in enumerate(s["master"] if c["master"] else s["params"]):
        n = p.numel()
        if c["bits"] == 8:
            of = torch.arange(n, device=DEV) // STATE_BLOCK
            m = s["m"][i].view(torch.float8_e4m3fn).double() * s["m_scale"][i].double()[of]
            v = s["v"][i].view(torch.float8_e5m2).double() * s["v_scale"][i].double()[of]
        else:
            m, v = s["m"][i].double(), s["v"][i].double()
        g = s["grads"][i].double()
        m = m.lerp(g, 1 - B1)
        v = v.lerp(g * g, 1 - B2)
        upd = (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + ADAM_EPS)
        new = p.double() - LR * WD * p.double() - LR * upd
        out["params"].append(new)
        if c["master"]:
            out["master"].append(new)
        if c["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
        else:
            idx = torch.nn.functional.pad(m, (0, -n % STATE_BLOCK)).view(-1, STATE_BLOCK)
            out["m_scale"].append(idx.abs().amax(1) / 448)
            idx = torch.nn.functional.pad(v, (0, -n % STATE_BLOCK)).view(-1, STATE_BLOCK)
            out["v_scale"].append(idx.amax(1) / 57344)
            out["m"].append(_round_e4m3(m / out["m_scale"][i][of]))
            out["v"].append(None)       # rounded at random: one of two neighbours
        del m, v, g, upd, new
    return out


def _round_e4m3(t):
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(t / step) * step).clamp(-448, 448)


def _exact_codes(v, rows):
    """(codes, scales) of v [rows, cols]: a scale and the quotients by it are held in 32 bits, by definition (a
    quotient of two 16-bit numbers often lies between two codes, and which is the nearer goes by that rounding)."""
    pad = torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).view(rows, -1, 128)
    top = pad.abs().amax(2)
    scale = torch.where(top > 0, top / 448, torch.ones_like(top)).float().double()
    return _round_e4m3((pad / scale[:, :, None]).float().double()).view(rows, -1)[:, :v.shape[1]], scale


def _spread(scale, shape):
    """A 128 x 128 block's scale at each element of a matrix."""
    r, c = (torch.arange(n, device=DEV) // 128 for n in shape)
    return scale.double()[..., r[:, None], c[None, :]]


def _exact_matmul(c, f):
    a, sa = _exact_codes(f["x"], c["M"])
    b = f["b"].view(torch.float8_e4m3fn).double() * _spread(f["bs"], f["b"].shape)
    return a, sa, (a * sa.repeat_interleave(128, 1)[:, :c["K"]]) @ b.T


def _exact_experts(c, f):
    R, I = c["T"] * c["K"], c["I"]
    a, sa = _exact_codes(f["x_disp"], R)
    x = a * sa.repeat_interleave(128, 1)
    y = torch.zeros(R, c["H"], dtype=torch.float64, device=DEV)
    at = f["offsets"].tolist()
    for e in range(c["E"]):
        if at[e] == at[e + 1]:
            continue
        rows = slice(at[e], at[e + 1])
        W1 = f["W1"][e].view(torch.float8_e4m3fn).double() * _spread(f["W1s"][e], f["W1"].shape[1:])
        W2 = f["W2"][e].view(torch.float8_e4m3fn).double() * _spread(f["W2s"][e], f["W2"].shape[1:])
        gu = x[rows] @ W1.T
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        q, sh = _exact_codes(h, at[e + 1] - at[e])
        y[rows] = (q * sh.repeat_interleave(128, 1)) @ W2.T
    return y * f["weight"][:, None]
