"""A whole layer for at most 8 tokens, against fp64.

The routing has to equal moe_router_topk's rule on fp64 logits (the inputs leave
gaps between them).  The output is held element by element to a bound that adds
up what the steps may be off:
  * an fp32 sum of products on the tensor cores keeps at least 13 bits of its
    largest term while aligning: 2^-13 S, S the sum of the terms' magnitudes;
  * with coded weights a token's value is represented within 2^-39 of its row's
    largest: r(x) = 2^-39 max|x|, none for bf16 weights;
  * |silu'| <= 1.1 and |silu(g)| <= |g|: h is off by 1.1 |u| dg + |g| du, and by 2^-11
    |h| for its rounding to f16 (half a step of 11 bits, at the most) with 2^-18 |h| for
    the exponential and the quotient;
  * h's small values: f16 has steps of 2^-24 below 2^-14, and the largest of eight
    columns is brought to 2^14 or more, so half a step is 2^-25 / 2^14 = 2^-39 of that
    largest; brought to the row's power of two (coded weights) a value is rounded so once
    more: r(h) = 2 * 2^-39 max|h| = 2^-38 max|h|;
  * a weight w_k moves by the logits' error, at most 2^-14 relative here;
  * the output's rounding: 2^-8 |out|.
"""
import ctypes

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_topk_multihot_gb300 as m
    return m


def make(moe, fmt, T, H, E, K, I, seed=0):
    """(x, router, kept W1, scales, kept W2, scales, the fp64 weights they stand for)."""
    g = torch.Generator(device=DEV).manual_seed(seed + T + H + E + K + I)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    x = (rnd(T, H) * torch.exp(rnd(T, 1))).bfloat16()
    router = rnd(E, H, std=H ** -0.5).bfloat16()
    W1, W2 = rnd(E, 2 * I, H, std=H ** -0.5).bfloat16(), rnd(E, H, I, std=I ** -0.5).bfloat16()
    if fmt == "bf16":
        return x, router, W1, None, W2, None, W1.double(), W2.double()
    if fmt == "fp8":
        (q1, s1), (q2, s2) = moe.moe_quantize_fp8_block(W1, 128), moe.moe_quantize_fp8_block(W2, 128)
        val = lambda q, s: (q.view(torch.float8_e4m3fn).double()  # noqa: E731
                            * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2))
    else:
        (q1, s1), (q2, s2) = moe.moe_quantize_fp4_block(W1), moe.moe_quantize_fp4_block(W2)
        val = lambda q, s: moe.moe_dequantize_fp4_block(q, s, torch.float32).double()  # noqa: E731
    return x, router, q1, s1, q2, s2, val(q1, s1), val(q2, s2)


def routing_of(x, router, K):
    logits = x.double() @ router.double().t()
    v, idx = logits.sort(dim=1, descending=True, stable=True)
    return idx[:, :K], torch.softmax(v[:, :K], 1)


def reference(x, idx, p, W1, W2, coded):
    """(fp64 output, its bound)."""
    T, H = x.shape
    I = W2.shape[2]
    rep = lambda v, r: r * v.abs().amax().expand(v.shape)  # noqa: E731
    out, lim = torch.zeros(T, H, dtype=torch.float64, device=x.device), torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for t in range(T):
        v = x[t].double()
        for e, w in {int(e): float(w) for e, w in zip(idx[t], p[t]) if e >= 0}.items():      # the last slot counts
            gu, d = W1[e] @ v, 2.0 ** -13 * (W1[e].abs() @ v.abs()) + W1[e].abs() @ rep(v, 2.0 ** -39 if coded else 0.0)
            g, u = gu[:I], gu[I:]
            h = g / (1 + torch.exp(-g)) * u
            dh = 1.1 * (u.abs() + d[I:]) * d[:I] + g.abs() * d[I:] + (2.0 ** -11 + 2.0 ** -18) * h.abs()
            o = W2[e] @ h
            do = W2[e].abs() @ dh + 2.0 ** -13 * (W2[e].abs() @ h.abs()) + W2[e].abs() @ rep(h, 2.0 ** -38)
            out[t] += w * o
            lim[t] += w * (do + 2.0 ** -14 * o.abs())
    return out, lim + 2.0 ** -8 * (out.abs() + lim)


def check(got, ref, lim):
    err = (got.double() - ref).abs()
    assert (err <= lim).all(), float((err / lim).max())
    rel = float(err.norm() / ref.norm())
    assert rel < 2.0 ** -9, rel       # the output's rounding, 2^-8 / sqrt(3) / sqrt(2) or so, hides the rest


# one token to eight; one expert and 1024; more h than tokens and the other way round;
# sizes where a CTA has no column of h or row of the output, several pieces of 16
# rows of it, a row shorter than a piece of the ring and one that ends inside it;
# h of all pairs in shared memory at once or not
SHAPES = [(1, 256, 8, 2, 128), (3, 256, 1, 1, 128), (8, 512, 8, 8, 384), (1, 2048, 128, 8, 768), (8, 2048, 128, 8, 768),
          (5, 768, 60, 6, 1024), (2, 8192, 4, 2, 128), (8, 256, 12, 3, 2048), (7, 1280, 1024, 16, 128), (4, 4096, 16, 4, 1280)]


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,H,E,K,I", SHAPES)
def test_layer(moe, fmt, T, H, E, K, I):
    x, router, W1, S1, W2, S2, V1, V2 = make(moe, fmt, T, H, E, K, I)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    buf = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)
    out, idx, p = moe.moe_layer_few(x, router, K, W1, W2, S1, S2, return_routing=True, out=buf[:T], status=status)
    assert (buf[T] == 7).all() and int(status) == 0
    ridx, rp = routing_of(x, router, K)
    assert torch.equal(idx, ridx)
    assert ((p.double() - rp).abs() <= 2.0 ** -14 * rp).all()
    check(out, *reference(x, ridx, rp, V1, V2, fmt != "bf16"))
    assert torch.equal(moe.moe_layer_few(x, router, K, W1, W2, S1, S2), out)          # and every order is fixed
    assert torch.equal(moe.moe_layer_few(x, router.float(), K, W1, W2, S1, S2), out)


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_given_routing(moe, fmt):
    T, H, E, K, I = 6, 512, 16, 4, 256
    x, router, W1, S1, W2, S2, V1, V2 = make(moe, fmt, T, H, E, K, I)
    idx = torch.tensor([[0, 15, 3, 7], [-1, -1, -1, -1], [2, 2, 2, 5], [1, -1, 1, -1], [9, 8, 9, 8], [4, 4, 4, 4]], device=DEV)
    p = torch.rand(T, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = moe.moe_layer_few(x, None, K, W1, W2, S1, S2, routing=(idx, p), status=status)
    ref, lim = reference(x, idx, p, V1, V2, fmt != "bf16")
    check(out, ref, lim)
    assert (out[1] == 0).all() and int(status) == 0
    # the same as the layer in several steps, within both roundings
    if fmt == "bf16":
        long = moe.moe_layer(x, idx, p, W1, W2)
        assert float((long.double() - ref).norm() / ref.norm()) < 2.0 ** -7
    bad = idx.clone()
    bad[0, 1], bad[3, 0] = E, -2
    want = idx.clone()
    want[0, 1], want[3, 0] = -1, -1
    got = moe.moe_layer_few(x, None, K, W1, W2, S1, S2, routing=(bad, p), status=status)
    assert int(status) == 1
    assert torch.equal(got, moe.moe_layer_few(x, None, K, W1, W2, S1, S2, routing=(want, p)))
    none = torch.full_like(idx, -1)
    assert (moe.moe_layer_few(x, None, K, W1, W2, S1, S2, routing=(none, p)) == 0).all()


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_unusual_values(moe, fmt):
    """A NaN or an infinity stays in its token's row; large, small and zero tokens; equal logits."""
    T, H, E, K, I = 8, 256, 8, 2, 128
    x, router, W1, S1, W2, S2, V1, V2 = make(moe, fmt, T, H, E, K, I)
    x[1, 7], x[2, 100] = float("nan"), float("inf")
    x[3] = 0
    x[4] *= 2.0 ** 40
    x[5] *= 2.0 ** -60
    x[6, 1:] *= 2.0 ** -30               # one value that dwarfs its neighbours
    out, idx, p = moe.moe_layer_few(x, router, K, W1, W2, S1, S2, return_routing=True)
    assert not torch.isfinite(out[1]).any() and not torch.isfinite(out[2]).any()
    assert idx[3].tolist() == [0, 1] and idx[1].tolist() == [0, 1] and (out[3] == 0).all()
    rest = [0, 4, 5, 6, 7]
    ridx, rp = routing_of(x[rest], router, K)
    assert torch.equal(idx[rest], ridx)
    ref, lim = reference(x[rest], ridx, p[rest].double(), V1, V2, fmt != "bf16")
    err = (out[rest].double() - ref).abs()
    # (2^-60 squared is in fp32's range; what lies below bf16's smallest normal number is off by its step)
    assert (err <= lim + 2.0 ** -133).all()


@gpu
def test_streams_graphs_and_two_at_once(moe):
    T, H, E, K, I = 2, 1024, 32, 4, 512
    sets = [make(moe, fmt, T, H, E, K, I, seed=9) for fmt in ("bf16", "fp8", "fp4")]
    want = [moe.moe_layer_few(s[0], s[1], K, s[2], s[4], s[3], s[5]) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[moe.moe_layer_few(s[0], s[1], K, s[2], s[4], s[3], s[5], stream=st) for s, st in zip(sets, streams)]
           for _ in range(20)]
    torch.cuda.synchronize()
    for row in got:
        assert all(torch.equal(a, b) for a, b in zip(row, want))
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = s[0]
            for _ in range(3):
                o = moe.moe_layer_few(o, s[1], K, s[2], s[4], s[3], s[5])
        graphs.append((g, o))
    for s in sets:
        s[0].copy_(-s[0])
    want = []
    for s in sets:
        o = s[0]
        for _ in range(3):
            o = moe.moe_layer_few(o, s[1], K, s[2], s[4], s[3], s[5])
        want.append(o)
    for _ in range(3):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for (_, o), w in zip(graphs, want))


def test_refusals_without_a_gpu(moe):
    from combine_topk_multihot_gb300 import _native as N
    p = 256

    def call(**kw):
        f = N.MoeFew(4, 8, 2, 256, 128, 0, 0, p, p, None, None, p, None, p, None, p, None, None, None, p)
        for k, v in kw.items():
            setattr(f, k, v)
        return N.lib.moe_layer_few(f, None)

    for kw in (dict(T=9), dict(E=0), dict(E=1025), dict(K=0), dict(K=9), dict(E=64, K=17), dict(H=0), dict(H=384), dict(I=0),
               dict(I=64), dict(T=8, H=16384), dict(T=8, I=16384), dict(T=1, H=131072)):
        assert call(**kw) == N.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(T=-1), dict(weights=3), dict(weights=-1), dict(router_dtype=2), dict(x=None), dict(W1=None), dict(W2=None),
               dict(out=None), dict(workspace=None), dict(router=None), dict(topk_idx=p), dict(router=None, topk_idx=p),
               dict(weights=1), dict(weights=2, W1_scale=p), dict(idx_out=p), dict(probs_out=p), dict(x=p + 8), dict(W1=p + 2),
               dict(router=p + 4), dict(workspace=p + 8), dict(out=p + 1), dict(weights=1, W1_scale=p + 2, W2_scale=p),
               dict(status=p + 2)):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert N.lib.moe_layer_few(None, None) == N.MOE_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert N.lib.moe_layer_few_workspace_bytes(9, 8, 2, 128, ctypes.byref(n)) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert N.lib.moe_layer_few_workspace_bytes(8, 8, 2, 128, None) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_layer_few_workspace_bytes(8, 8, 2, 128, ctypes.byref(n)) == 0 and n.value == 256 + 256 + 8 * 2 * 128 // 8 * 17


@gpu
def test_refusals(moe):
    T, H, E, K, I = 2, 256, 8, 2, 128
    x, router, W1, S1, W2, S2, *_ = make(moe, "fp4", T, H, E, K, I)
    ok = dict(x=x, router=router, top_k=K, W1=W1, W2=W2, W1_scale=S1, W2_scale=S2)
    assert moe.moe_layer_few(**ok).shape == (T, H)
    assert moe.moe_layer_few(**{**ok, "x": x[:0]}).shape == (0, H)
    idx, p = torch.zeros(T, K, dtype=torch.int64, device=DEV), torch.zeros(T, K, device=DEV)
    for kw, err in ((dict(x=x.float()), TypeError), (dict(x=x.cpu()), ValueError), (dict(x=x[:, ::2]), ValueError),
                    (dict(W2_scale=None), ValueError), (dict(router=None), ValueError), (dict(routing=(idx, p)), ValueError),
                    (dict(router=router.half()), TypeError), (dict(router=router[:4]), ValueError),
                    (dict(router=None, routing=(idx.int(), p)), TypeError), (dict(W1=W1.view(E, -1, H)), ValueError),
                    (dict(W1_scale=S1.float(), W2_scale=S2.float()), ValueError), (dict(W1_scale=None, W2_scale=None), TypeError),
                    (dict(top_k=9), moe.MoEError), (dict(x=x.repeat(5, 1)), moe.MoEError)):
        with pytest.raises(err):
            moe.moe_layer_few(**{**ok, **kw})


# ------------------------------------------------------------------ through the operators and the block
def _meta(T=3, H=256, E=8, K=2, I=128):
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="meta")  # noqa: E731
    u8 = lambda *s: mk(*s, dt=torch.uint8)  # noqa: E731
    return dict(x=mk(T, H), normed=mk(T, H), router=mk(E, H), W1=mk(E, 2 * I, H), W2=mk(E, H, I), w=mk(H, dt=torch.float32),
                q1=u8(E, 2 * I, H // 2), s1=u8(E, 2 * I // 128, H // 128, 32, 4, 4), q2=u8(E, H, I // 2),
                s2=u8(E, H // 128, I // 128, 32, 4, 4))


def _used(fn, *a):
    from torch.fx.experimental.proxy_tensor import make_fx
    gm = make_fx(fn)(*a)
    return {str(n.target).split(".")[1] for n in gm.graph.nodes if str(n.target).startswith("moe_gb300.")}


def test_block_takes_the_short_way_without_a_gpu(moe):
    """Which operators a block goes through, by tokens, weights, `few` and wanted gradients."""
    short, plain = {"layer_few", "norm_out"}, {"router_topk", "route_to_multihot", "dispatch", "grouped_experts", "combine", "norm_out"}
    for T in (1, 8, 9):
        t = _meta(T)
        run = lambda W1, W2, **kw: moe.moe_block(t["x"], t["normed"], t["router"], 2, W1, W2, t["w"], **kw)[0]  # noqa: E731
        bf = (t["W1"], t["W2"])
        assert _used(lambda *a: run(*a), *bf) == plain
        assert _used(lambda *a: run(*a, few=True), *bf) == (short if T <= 8 else plain)
        assert _used(lambda q1, q2: run(q1, q2, fp4=(t["s1"], t["s2"])), t["q1"], t["q2"]) == (
            short if T <= 8 else plain | {"dequantize_fp4_block"})
        grad = t["normed"].clone().requires_grad_()
        block = lambda n, W1, W2, **kw: moe.moe_block(t["x"], n, t["router"], 2, W1, W2, t["w"], **kw)[0]  # noqa: E731
        assert block(grad, *bf, few=True).requires_grad
        out = block(grad, t["q1"], t["q2"], fp4=(t["s1"], t["s2"]))
        out.float().sum().backward()
        assert grad.grad.shape == grad.shape
        with torch.no_grad():
            assert _used(lambda n: block(n, *bf, few=True), grad.detach()) == (short if T <= 8 else plain)
    with pytest.raises(ValueError, match="not both"):
        moe.moe_block(t["x"], t["normed"], t["router"], 2, t["q1"], t["q2"], t["w"], fp8=(1, 2), fp4=(1, 2))
    assert moe.moe_layer_few_fits(8, 128, 8, 2048, 768) and not moe.moe_layer_few_fits(9, 128, 8, 2048, 768)
    assert not moe.moe_layer_few_fits(8, 128, 8, 2048, 8192) and moe.moe_layer_few_fits(8, 128, 8, 2048, 7168, _meta()["s1"])
    ns = torch.ops.moe_gb300
    c, s = ns.quantize_fp4_block(torch.zeros(3, 200, 160, device="meta"))
    assert c.shape == (3, 200, 80) and s.shape == (3, 2, 2, 32, 4, 4) and ns.dequantize_fp4_block(c, s).shape == (3, 200, 160)
    with pytest.raises(NotImplementedError, match="CPU"):
        ns.quantize_fp4_block(torch.zeros(4, 64))


@pytest.mark.parametrize("dynamic", [None, False, True])
def test_block_compiles_as_one_graph_without_a_gpu(moe, dynamic):
    t = _meta(8)
    blocks = (lambda x, n: moe.moe_block(x, n, t["router"], 2, t["W1"], t["W2"], t["w"], few=True)[0],
              lambda x, n: moe.moe_block(x, n, t["router"], 2, t["q1"], t["q2"], t["w"], fp4=(t["s1"], t["s2"]))[0])
    for block in blocks:
        torch._dynamo.reset()
        compiled = torch.compile(block, fullgraph=True, backend="aot_eager", dynamic=dynamic)
        with torch.no_grad():
            for T in (1, 3, 8, 9, 40):
                x = torch.zeros(T, t["x"].shape[1], dtype=torch.bfloat16, device="meta")
                assert compiled(x, x).shape == x.shape
    torch._dynamo.reset()


def test_block_with_another_router_type_takes_the_long_way_without_a_gpu(moe):
    t = _meta(4)
    run = lambda r: moe.moe_block(t["x"], t["normed"], r, 2, t["W1"], t["W2"], t["w"], few=True)[0]  # noqa: E731
    assert "layer_few" in _used(run, t["router"].float()) and "layer_few" not in _used(run, t["router"].half())


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_block(moe, fmt):
    """A block for a few tokens against the same block of more tokens, whose first rows they are."""
    H, E, K, I = 512, 16, 4, 256
    x, router, W1, S1, W2, S2, V1, V2 = make(moe, fmt, 8, H, E, K, I)
    g = torch.Generator(device=DEV).manual_seed(1)
    many, (w, w2) = torch.randn(40, H, generator=g, device=DEV).bfloat16(), torch.rand(2, H, generator=g, device=DEV) + 0.5
    gate = torch.randn(40, generator=g, device=DEV)
    kw = {} if fmt == "bf16" else {fmt: (S1, S2)}
    normed, _ = torch.ops.moe_gb300.norm_in(many, w, 1e-6, 0.0)
    whole = moe.moe_block(many, normed, router, K, W1, W2, w, gate=gate, next_weight=w2, return_status=True, **kw)
    for T in (1, 5, 8):
        few = moe.moe_block(many[:T], normed[:T], router, K, W1, W2, w, gate=gate[:T], next_weight=w2, return_status=True, few=True, **kw)
        assert int(few[2]) == 0
        for a, b in zip(few[:2], whole[:2]):
            rel = float((a.double() - b[:T].double()).norm() / b[:T].double().norm())
            # the layer's own roundings: e4m3 activations (2^-4, two of them) in moe_layer_fp8_block, bf16 in the others
            assert rel < (2.0 ** -4 if fmt == "fp8" else 2.0 ** -7), rel
    if fmt == "fp4":
        idx, p = torch.ops.moe_gb300.router_topk((normed.float() @ router.float().t()).contiguous(), K)
        long, st = moe.moe_layer_fp4_block(normed, idx, p, W1, S1, W2, S2, return_status=True)
        assert torch.equal(long, moe.moe_layer(normed, idx, p, moe.moe_dequantize_fp4_block(W1, S1), moe.moe_dequantize_fp4_block(W2, S2)))
        short = moe.moe_layer_fp4_block(normed[:8], idx[:8], p[:8], W1, S1, W2, S2)
        assert torch.equal(short, moe.moe_layer_few(normed[:8], None, K, W1, W2, S1, S2, routing=(idx[:8], p[:8])))
        assert float((short.double() - long[:8].double()).norm() / long[:8].double().norm()) < 2.0 ** -7


@gpu
def test_opcheck(moe):
    ns, tests = torch.ops.moe_gb300, ("test_schema", "test_autograd_registration", "test_faketensor", "test_aot_dispatch_dynamic")
    x, router, W1, S1, W2, S2, *_ = make(moe, "fp4", 3, 256, 8, 2, 128)
    idx, p = routing_of(x, router, 2)
    torch.library.opcheck(ns.layer_few.default, (x, router, None, None, 2, W1, W2, S1, S2), test_utils=tests)
    torch.library.opcheck(ns.layer_few.default, (x, None, idx, p.float(), 2, W1, W2, S1, S2), test_utils=tests)
    a = torch.randn(9, 160, device=DEV)
    q, s = ns.quantize_fp4_block(a)
    torch.library.opcheck(ns.quantize_fp4_block.default, (a,), test_utils=tests)
    torch.library.opcheck(ns.dequantize_fp4_block.default, (q, s), test_utils=tests)
    torch.library.opcheck(ns.matmul_fp4_block.default, (q, s, q, s), test_utils=tests)


@gpu
def test_another_device_is_refused(moe, monkeypatch):
    from combine_topk_multihot_gb300 import moe as core
    x, router, W1, S1, W2, S2, *_ = make(moe, "fp4", 3, 256, 8, 2, 128)
    q, s = moe.moe_quantize_fp4_block(x)
    now = torch.cuda.current_device()
    monkeypatch.setattr(core, "_current_device", lambda: now + 1)
    for call in (lambda: moe.moe_quantize_fp4_block(x), lambda: moe.moe_dequantize_fp4_block(q, s),
                 lambda: moe.moe_matmul_fp4_block(q, s, q, s), lambda: moe.moe_layer_few(x, router, 2, W1, W2, S1, S2)):
        with pytest.raises(ValueError, match="current device"):
            call()


@gpu
@pytest.mark.parametrize("ctas", [0, 7])
def test_a_meeting_that_fails(moe, ctas):
    """CTAs that do not come to the meeting: about 2 s, then a status and NaN; the next call is whole again."""
    x, router, W1, S1, W2, S2, *_ = make(moe, "fp8", 3, 256, 8, 2, 128)
    whole = moe.moe_layer_few(x, router, 2, W1, W2, S1, S2)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib = moe._native.lib
    try:
        assert lib.moe_selftest_few_ctas(ctas) == 0
        out = moe.moe_layer_few(x, router, 2, W1, W2, S1, S2, status=status)
    finally:
        assert lib.moe_selftest_few_ctas(-1) == 0
    torch.cuda.synchronize()
    assert out.isnan().all() and int(status) == moe._native.MOE_DEVERR_TIMEOUT
    assert torch.equal(moe.moe_layer_few(x, router, 2, W1, W2, S1, S2), whole)


# the two kinds of CTA and all widths: no tile arrives, or the first of each CTA's
@gpu
@pytest.mark.parametrize("M,N,K,tiles", [(100, 520, 512, 0), (100, 513, 512, 0), (300, 513, 96, 0), (1000, 4096, 384, 0),
                                         (2049, 4096, 256, 0), (5000, 8192, 384, 1), (4100, 8195, 384, 1)])
def test_a_product_whose_operands_stop(moe, M, N, K, tiles):
    g = torch.Generator(device=DEV).manual_seed(M)
    a, b = (moe.moe_quantize_fp4_block(torch.randn(n, K, generator=g, device=DEV)) for n in (M, N))
    whole = moe.moe_matmul_fp4_block(*a, *b)
    lib = moe._native.lib
    status, out = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    try:
        assert lib.moe_selftest_block_product_tiles(tiles) == 0
        moe.moe_matmul_fp4_block(*a, *b, out=out, status=status)
    finally:
        assert lib.moe_selftest_block_product_tiles(-1) == 0
    torch.cuda.synchronize()
    missing = out.isnan()
    assert missing.all() if tiles == 0 else missing.any() and not missing.all()
    assert torch.equal(out[~missing], whole[~missing]) and int(status) == moe._native.MOE_DEVERR_TIMEOUT
    assert torch.equal(moe.moe_matmul_fp4_block(*a, *b), whole)


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("apart", [16, 26, 27])
def test_columns_of_h_far_below_others(moe, fmt, apart):
    """Columns of h around 2^apart below others of their row, which W2 multiplies by zero: with codes they
    still are exact down to 2^-28 of the row's largest, and never off by more than 2^-38 of it."""
    T, H, E, K, I = 3, 256, 2, 1, 256
    g = torch.Generator(device=DEV).manual_seed(apart)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    x, W1, W2 = rnd(T, H).bfloat16(), rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5)
    W1[:, I:I + 128] *= 2.0 ** apart     # up rows of the first 128 columns
    W2[:, :, :128] = 0
    W1, W2, S1, S2 = W1.bfloat16(), W2.bfloat16(), None, None
    V1, V2 = W1.double(), W2.double()
    if fmt != "bf16":
        quantize = (lambda w: moe.moe_quantize_fp8_block(w, 128)) if fmt == "fp8" else moe.moe_quantize_fp4_block
        (W1, S1), (W2, S2) = quantize(W1), quantize(W2)
        if fmt == "fp8":
            V1, V2 = (q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
                      for q, s in ((W1, S1), (W2, S2)))
        else:
            V1, V2 = (moe.moe_dequantize_fp4_block(q, s, torch.float32).double() for q, s in ((W1, S1), (W2, S2)))
    idx, p = torch.tensor([[0], [1], [0]], device=DEV), torch.ones(T, K, device=DEV)
    out = moe.moe_layer_few(x, None, K, W1, W2, S1, S2, routing=(idx, p))
    ref, lim = reference(x, idx, p, V1, V2, fmt != "bf16")
    err = (out.double() - ref).abs()
    assert (err <= lim).all(), float((err / lim).max())
    assert float(lim.norm() / ref.norm()) < 0.25       # (columns that were lost would show)


# layers of which h does not lie in shared memory at once: with several groups of 16 rows of the output a CTA
# h is brought again for each, in parts, and two pieces a warp are the fewest
LARGE = [(8, 4096, 32, 8, 1536), (8, 7168, 16, 8, 2048), (3, 16384, 8, 4, 2048)]


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_large_shapes_reach_every_way_of_bringing_h_without_a_gpu(moe, fmt):
    from combine_topk_multihot_gb300 import _native as N
    seen = set()
    for T, H, E, K, I in SHAPES + LARGE:
        rows, slots = ctypes.c_int32(), ctypes.c_int32()
        assert N.lib.moe_selftest_few_plan(T, K, H, I, fmt, ctypes.byref(rows), ctypes.byref(slots)) == 0
        assert T <= rows.value <= T * K and 2 <= slots.value <= 6
        seen.add(("whole" if rows.value == T * K else "parts", "one group" if H <= 152 * 16 else "groups"))
        seen.add(slots.value)
    assert {("whole", "one group"), ("whole", "groups"), ("parts", "groups"), 2} <= seen, seen
    out = ctypes.byref(ctypes.c_int32())
    assert N.lib.moe_selftest_few_plan(8, 8, 16384, 128, fmt, out, out) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_selftest_few_plan(8, 8, 256, 128, fmt, None, out) == N.MOE_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,H,E,K,I", LARGE)
def test_large_layer(moe, fmt, T, H, E, K, I):
    test_layer(moe, fmt, T, H, E, K, I)
