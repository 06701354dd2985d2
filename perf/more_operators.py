"""Serving a layer's experts to a few tokens, and 4-bit weights, as measured cases.

Three kinds of pass.  ``quantize``: values to microscaled 4-bit floating point
(e2m1 codes, two a byte, a power-of-two scale for each 32 of a row) and back to
bf16.  ``matmul``: the dense product of such codes, from bf16 rows.  ``layer``: a
whole mixture-of-experts layer (router, top-k, SwiGLU experts, weighted sum) for
at most 8 tokens, from bf16 weights, e4m3 codes with a scale per 128 x 128
block, or 4-bit codes.
"""
import math

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # the activations of a few decoded tokens
        dict(name="quantize 7", kind="quantize", batch=1, rows=7, cols=2048, src="bf16"),
        # a ragged prompt batch of an fp32 stream, rows of an odd number of blocks
        dict(name="quantize 333", kind="quantize", batch=1, rows=333, cols=4000, src="fp32"),
        # the gate/up weights of 128 experts, H=2048, I=768
        dict(name="quantize weights", kind="quantize", batch=128, rows=1536, cols=2048, src="bf16"),
        # a projection of a few decoded tokens
        dict(name="matmul 7", kind="matmul", M=7, N=4096, K=2048),
        # a projection of a ragged batch, with odd sizes
        dict(name="matmul 333", kind="matmul", M=333, N=4097, K=2080),
        # a projection of a ragged prompt batch
        dict(name="matmul 4097", kind="matmul", M=4097, N=4096, K=4096),
        # a wide projection of a long prompt batch
        dict(name="matmul 8192", kind="matmul", M=8192, N=8192, K=4096),
        # one decoded token through its 8 of 128 experts in bf16
        dict(name="layer bf16 1", kind="layer", w="bf16", T=1, H=2048, E=128, K=8, I=768),
        # the same from 4-bit weights
        dict(name="layer fp4 1", kind="layer", w="fp4", T=1, H=2048, E=128, K=8, I=768),
        # a small batch of decoded tokens from e4m3 weights
        dict(name="layer fp8 5", kind="layer", w="fp8", T=5, H=2048, E=128, K=8, I=768),
        # a full batch of decoded tokens in bf16
        dict(name="layer bf16 8", kind="layer", w="bf16", T=8, H=2048, E=128, K=8, I=768),
        # few wide experts from 4-bit weights
        dict(name="layer fp4 8", kind="layer", w="fp4", T=8, H=4096, E=16, K=4, I=1280),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "matmul", "layer"])
    if kind == "quantize":
        batch, cols = rng.choice([1, 1, 1, 4, 16]), 32 * _log(rng, 1, 256)
        rows = max(1, min(_log(rng, 1, 16384), 400_000_000 // (batch * cols)))
        return dict(kind=kind, batch=batch, rows=rows, cols=cols, src=rng.choice(["bf16", "fp32"]))
    if kind == "matmul":
        N, K = _log(rng, 64, 8192), 32 * _log(rng, 4, 256)
        M = max(1, min(_log(rng, 1, 8192), 8192 * 8192 * 4096 // (N * K)))
        return dict(kind=kind, M=M, N=N, K=K)
    E = rng.choice([8, 16, 32, 64, 128])
    return dict(kind=kind, w=rng.choice(["bf16", "fp8", "fp4"]), T=rng.randint(1, 8), H=256 * rng.randint(1, 8), E=E,
                K=rng.choice([1, 2, 4, 6, 8]), I=128 * rng.randint(1, 6))


# ---------------------------------------------------------------- the inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["kind"] == "quantize":
        # rows of different size, as activations and trained weights have them
        std = torch.rand(c["batch"], c["rows"], 1, generator=g, device=DEV) + 0.5
        return dict(case=c, src=(_randn(g, c["batch"], c["rows"], c["cols"]) * std).to(_TYPES[c["src"]]))
    if c["kind"] == "matmul":
        b, bs = _quantize(_randn(g, c["N"], c["K"], std=0.02))
        return dict(case=c, x=_randn(g, c["M"], c["K"], dtype=torch.bfloat16), b=b, bs=bs)
    T, H, E, I = c["T"], c["H"], c["E"], c["I"]
    s = dict(case=c, x=_randn(g, T, H, dtype=torch.bfloat16), router=_randn(g, E, H, dtype=torch.bfloat16, std=H ** -0.5))
    for name, shape in (("W1", (2 * I, H)), ("W2", (H, I))):
        made = [_weights(c["w"], _randn(g, *shape, std=shape[1] ** -0.5)) for _ in range(E)]
        s[name] = torch.stack([m[0] for m in made])
        s[name + "s"] = None if made[0][1] is None else torch.stack([m[1] for m in made])
    return s


def _weights(kind, w):
    """A matrix as it is kept: (values or codes, scales or None)."""
    if kind == "bf16":
        return w.bfloat16(), None
    if kind == "fp4":
        return _quantize(w)
    R, C = w.shape
    b = w.view(R // 128, 128, C // 128, 128)
    scale = b.abs().amax((1, 3)) / 448
    return (b / scale[:, None, :, None]).view(R, C).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _blocks(v):
    """(|v| and its signs in blocks of 32, the blocks' e8m0 scales as their 8 bits)."""
    b = v.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    # the exponent of the largest value less 2, one more where it is 7/4 of a power of two or above
    e = (((top.view(torch.int32) + (1 << 21)) >> 23) - 2).clamp_min(0)
    return b, torch.where(top.isfinite(), e, 255)


def _quantize(v):
    """e2m1 codes of v [..., rows, cols], two a byte, the lower four bits first; the scales in tiles."""
    b, e = _blocks(v)
    q = (b * torch.exp2(127.0 - e)[..., None]).abs()
    code = (q > 0.25).int() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5)
    code = (code | torch.where(torch.signbit(b), 8, 0)).to(torch.uint8).flatten(-2)
    return code[..., ::2] | code[..., 1::2] << 4, _tiles(e.to(torch.uint8))


def _tiles(s):
    """Scales [..., rows, blocks] as tiles of 128 rows x 4 blocks [..., row tiles, block tiles, 32, 4, 4]: row r of a
    tile lies at [r % 32, r / 32]; zeros past the edges."""
    R, B = s.shape[-2:]
    s = torch.nn.functional.pad(s, (0, -B % 4, 0, -R % 128))
    s = s.view(*s.shape[:-2], (R + 127) // 128, 4, 32, (B + 3) // 4, 4)
    return s.movedim(-2, -4).transpose(-3, -2).contiguous()


def _untile(t, R, B):
    s = t.transpose(-3, -2).movedim(-4, -2)
    return s.reshape(*s.shape[:-5], s.shape[-5] * 128, s.shape[-2] * 4)[..., :R, :B]


def _values(codes, scales):
    """What codes and tiled scales stand for, in fp32."""
    R, C = codes.shape[-2], codes.shape[-1] * 2
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    m = n & 7
    # 0 and 0.5, else (1 or 1.5) times 1, 2 or 4
    v = torch.where(m < 2, m * 0.5, (2 + (m & 1)) * torch.exp2((m >> 1) - 2.0))
    v = torch.where(n > 7, -v, v).unflatten(-1, (-1, 32))
    e = _untile(scales, R, C // 32).float()
    scale = torch.where(e == 255, float("nan"), torch.exp2(e - 127))
    return (v * scale[..., None]).flatten(-2)


# -------------------------------------------------------------------- a pass
def run(state):
    k = state["case"]["kind"]
    if own:
        import combine_topk_multihot_gb300 as moe
        return {"quantize": _own_quantize, "matmul": _own_matmul, "layer": _own_layer}[k](moe, state)
    return {"quantize": _plain_quantize, "matmul": _plain_matmul, "layer": _plain_layer}[k](state)


def _own_quantize(moe, s):
    codes, scales = moe.moe_quantize_fp4_block(s["src"])
    return moe.moe_dequantize_fp4_block(codes, scales), scales.view(torch.float8_e8m0fnu)


def _own_matmul(moe, s):
    a, a_scale = moe.moe_quantize_fp4_block(s["x"])
    return moe.moe_matmul_fp4_block(a, a_scale, s["b"], s["bs"])


def _own_layer(moe, s):
    return moe.moe_layer_few(s["x"], s["router"], s["case"]["K"], s["W1"], s["W2"], W1_scale=s["W1s"], W2_scale=s["W2s"])


def _plain_quantize(s):
    codes, scales = _quantize(s["src"])
    return _values(codes, scales).bfloat16(), scales.view(torch.float8_e8m0fnu)


def _plain_matmul(s):
    return (_values(*_quantize(s["x"])) @ _values(s["b"], s["bs"]).t()).bfloat16()


def _expert(s, name, idx):
    """The chosen experts' matrices [T, K, rows, cols] in fp32."""
    w, scale = s[name][idx], s[name + "s"]
    if scale is None:
        return w.float()
    if scale.dtype == torch.uint8:
        return _values(w, scale[idx])
    f = scale[idx].repeat_interleave(128, -1).repeat_interleave(128, -2)
    return w.view(torch.float8_e4m3fn).float() * f


def _plain_layer(s):
    c, x = s["case"], s["x"].float()
    logits, idx = (x @ s["router"].float().t()).sort(dim=1, descending=True, stable=True)
    p = torch.exp(logits - logits[:, :1])[:, :c["K"]]
    p, idx = p / p.sum(1, keepdim=True), idx[:, :c["K"]]
    gu = _expert(s, "W1", idx) @ x[:, None, :, None]
    g, u = gu[:, :, :c["I"]], gu[:, :, c["I"]:]
    h = g / (1 + torch.exp(-g)) * u
    return ((_expert(s, "W2", idx) @ h).squeeze(-1) * p[:, :, None]).sum(1).bfloat16()


# -------------------------------------------------------- the work of a pass
def work(case):
    c = case
    if c["kind"] == "quantize":
        n = c["batch"] * c["rows"] * c["cols"]
        return dict(bytes=n * (2 if c["src"] == "bf16" else 4) + n // 32 + n * 2, flops=n * 4)
    if c["kind"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(bytes=M * K * 2 + N * K // 2 + N * K // 32 + M * N * 2, flops=2 * M * N * K)
    T, H, E, K, I = c["T"], c["H"], c["E"], c["K"], c["I"]
    used = E * (1 - (1 - K / E) ** T)       # experts that get a token
    each = {"bf16": 2, "fp8": 1 + 4 / 128 ** 2, "fp4": 0.5 + 1 / 32}[c["w"]]
    return dict(bytes=int(used * 3 * H * I * each + E * H * 2 + T * H * 4), flops=T * (6 * K * H * I + 2 * E * H))


# ---------------------------------------------- the same from 64-bit formulas
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "matmul": _exact_matmul, "layer": _exact_layer}[case["kind"]](case, s)


def _exact_codes(v):
    """(the nearest e2m1 values, the scales) of v [rows, cols] in blocks of 32; midway the one with an even code."""
    b = v.double().view(v.shape[0], -1, 32)
    top = b.abs().max(-1).values
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -126))) - 2
    scale = torch.exp2((e + (top >= 7 * torch.exp2(e))).clamp_min(-127))
    scale = torch.where(top == 0, 2.0 ** -127, scale)
    q, best = (b / scale[..., None]).abs(), torch.zeros_like(b)
    for i in range(1, 8):
        mid = (_E2M1[i - 1] + _E2M1[i]) / 2
        best = torch.where((q > mid) | ((q == mid) & (i % 2 == 0)), _E2M1[i], best)
    return torch.copysign(best, b), scale


def _exact_quantize(c, s):
    R, B = c["rows"], c["cols"] // 32
    q, scale = _exact_codes(s["src"].view(-1, c["cols"]))
    tiles = torch.full((c["batch"], -(-R // 128) * 128, -(-B // 4) * 4), 2.0 ** -127, dtype=torch.float64, device=DEV)
    tiles[:, :R, :B] = scale.view(c["batch"], R, B)
    row, col = torch.arange(tiles.shape[1], device=DEV), torch.arange(tiles.shape[2], device=DEV)
    out = torch.empty(c["batch"], -(-R // 128), -(-B // 4), 32, 4, 4, dtype=torch.float64, device=DEV)
    out[:, (row // 128)[:, None], (col // 4)[None], (row % 32)[:, None], (row % 128 // 32)[:, None], (col % 4)[None]] = tiles
    return (q * scale[..., None]).view(c["batch"], R, c["cols"]), out


def _exact_weights(w, scale):
    """One matrix in 64 bits."""
    if scale is None:
        return w.double()
    if scale.dtype == torch.float32:
        r, c = (torch.arange(n, device=DEV) // 128 for n in w.shape)
        return w.view(torch.float8_e4m3fn).double() * scale.double()[r[:, None], c[None]]
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=DEV)
    v = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=DEV)
    v[:, 0::2], v[:, 1::2] = table[(w % 16).long()], table[(w // 16).long()]
    r, b = torch.arange(v.shape[0], device=DEV)[:, None], (torch.arange(v.shape[1], device=DEV) // 32)[None]
    return v * torch.exp2(scale[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].double() - 127)


def _exact_matmul(c, s):
    q, scale = _exact_codes(s["x"])
    a = (q * scale[..., None]).view(c["M"], c["K"])
    b = _exact_weights(s["b"], s["bs"])
    return a @ b.T


def _exact_layer(c, s):
    x, I = s["x"].double(), c["I"]
    logits = torch.einsum("th,eh->te", x, s["router"].double())
    out = torch.zeros_like(x)
    for t in range(c["T"]):
        best, chosen = logits[t].topk(c["K"])
        for e, p in zip(chosen.tolist(), torch.softmax(best, 0)):
            scales = [None if s[n] is None else s[n][e] for n in ("W1s", "W2s")]
            gu = _exact_weights(s["W1"][e], scales[0]) @ x[t]
            out[t] += p * (_exact_weights(s["W2"][e], scales[1]) @ (gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]))
    return out
