"""Gradients through experts whose weights get none: bf16 weights that want no gradient,
and e2m1 codes, which can have none.

The weights' gradients are neither computed nor is anything kept for them, and the
others are the same bit for bit as beside them.  Against fp64 a gradient passes at most
six roundings to bf16 (the gate and up values, h, the output before its weight, the weighted
gradient, that of the gate and up values, the row's and the sum's), each at most 2^-8
relative to its element; the sums in between are of independent terms, so that a
relative error carries over to their norm: 6 * 2^-8 of the gradient's norm together.
"""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_topk_multihot_gb300 as m
    return m


class _Used(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.ops = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.namespace == "moe_gb300":
            self.ops.add(func._opname)
        return func(*args, **(kwargs or {}))


def _meta(T=40, H=256, E=8, K=2, I=128):
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="meta")  # noqa: E731
    u8 = lambda *s: mk(*s, dt=torch.uint8)  # noqa: E731
    return dict(x=mk(T, H), idx=mk(T, K, dt=torch.int64), p=mk(T, K, dt=torch.float32), W1=mk(E, 2 * I, H), W2=mk(E, H, I),
                q1=u8(E, 2 * I, H // 2), s1=u8(E, 2 * I // 128, H // 128, 32, 4, 4), q2=u8(E, H, I // 2),
                s2=u8(E, H // 128, I // 128, 32, 4, 4))


@pytest.mark.parametrize("T", [3, 40])
def test_codes_keep_and_compute_nothing_for_their_gradients_without_a_gpu(moe, T):
    t, kept = _meta(T), []
    x, p = t["x"].requires_grad_(), t["p"].requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(lambda v: kept.append((tuple(v.shape), v.dtype)) or v, lambda v: v):
        out = moe.moe_layer_fp4_block(x, t["idx"], p, t["q1"], t["s1"], t["q2"], t["s2"])
    assert not {s for s, d in kept if d is torch.bfloat16 and len(s) == 3}         # no weights as values
    assert {(tuple(t[k].shape), torch.uint8) for k in ("q1", "s1", "q2", "s2")} <= set(kept)
    with _Used() as used:
        gx, gp = torch.autograd.grad(out, (x, p), torch.zeros_like(out))
    assert gx.shape == x.shape and gx.dtype is torch.bfloat16 and gp.shape == p.shape and gp.dtype is torch.float32
    assert used.ops == {"combine_backward", "dequantize_fp4_block", "experts_backward_rows", "dispatch_backward",
                        "route_to_multihot_backward"}


@pytest.mark.parametrize("wanted", ["", "W1", "W2", "W1 W2"])
def test_weights_that_want_no_gradient_without_a_gpu(moe, wanted):
    t = _meta()
    t["x"].requires_grad_()
    for k in wanted.split():
        t[k].requires_grad_()
    out = moe.moe_layer(t["x"], t["idx"], t["p"], t["W1"], t["W2"])
    with _Used() as used:
        out.float().sum().backward()
    assert ("experts_backward" in used.ops) == bool(wanted) and ("experts_backward_rows" in used.ops) == (not wanted)
    for k in ("W1", "W2"):
        g = t[k].grad
        assert (g is None) if k not in wanted else (g.shape == t[k].shape and g.dtype is t[k].dtype)
    assert t["x"].grad.shape == t["x"].shape and t["p"].grad is None


def test_compiles_as_one_graph_without_a_gpu(moe):
    t = _meta()
    x, p = t["x"].requires_grad_(), t["p"].requires_grad_()
    for layer in (lambda x, p: moe.moe_layer(x, t["idx"], p, t["W1"], t["W2"]),
                  lambda x, p: moe.moe_layer_fp4_block(x, t["idx"], p, t["q1"], t["s1"], t["q2"], t["s2"])):
        torch._dynamo.reset()
        out = torch.compile(layer, fullgraph=True, backend="aot_eager")(x, p)
        gx, gp = torch.autograd.grad(out, (x, p), torch.zeros_like(out))
        assert gx.shape == x.shape and gp.shape == p.shape
    torch._dynamo.reset()


def _exact(x, idx, p, W1, W2):
    """The layer in fp64, differentiable; of an expert that a token names twice the last slot counts."""
    T, K = idx.shape
    I = W2.shape[2]
    rows = []
    for t in range(T):
        out = torch.zeros_like(x[0])
        for e, k in {int(idx[t, k]): k for k in range(K) if idx[t, k] >= 0}.items():
            gu = W1[e] @ x[t]
            out = out + p[t, k] * (W2[e] @ (torch.nn.functional.silu(gu[:I]) * gu[I:]))
        rows.append(out)
    return torch.stack(rows)


def _case(moe, T, seed=0):
    H, E, K, I = 512, 8, 3, 256
    g = torch.Generator(device=DEV).manual_seed(seed + T)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    idx = torch.rand(T, E, generator=g, device=DEV).topk(K, dim=1).indices
    idx[0, 1], idx[T - 1, 0] = -1, idx[T - 1, 2]           # no expert; one named twice
    return (rnd(T, H).bfloat16(), idx, torch.rand(T, K, generator=g, device=DEV), rnd(E, 2 * I, H, std=H ** -0.5),
            rnd(E, H, I, std=I ** -0.5), rnd(T, H).bfloat16())


@gpu
@pytest.mark.parametrize("pad", [1, 64])
@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_gradients_through_codes(moe, T, pad):
    x, idx, p, W1, W2, grad = _case(moe, T)
    (q1, s1), (q2, s2) = moe.moe_quantize_fp4_block(W1), moe.moe_quantize_fp4_block(W2)
    V1, V2 = moe.moe_dequantize_fp4_block(q1, s1), moe.moe_dequantize_fp4_block(q2, s2)
    x.requires_grad_(), p.requires_grad_()
    out = moe.moe_layer_fp4_block(x, idx, p, q1, s1, q2, s2, pad)
    got = torch.autograd.grad(out, (x, p), grad, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(out, (x, p), grad), got))
    # beside the weights' gradients, bit for bit
    t1, t2 = V1.clone().requires_grad_(), V2.clone().requires_grad_()
    full = torch.autograd.grad(moe.moe_layer(x, idx, p, t1, t2, pad), (x, p, t1, t2), grad)
    assert torch.equal(out, moe.moe_layer(x, idx, p, V1, V2, pad)) and all(torch.equal(a, b) for a, b in zip(got, full))
    # against the formula's gradients, and those against differences
    xd, pd = x.detach().double().requires_grad_(), p.detach().double().requires_grad_()
    f = lambda a, b: (_exact(a, idx, b, V1.double(), V2.double()) * grad.double()).sum()  # noqa: E731
    ref = torch.autograd.grad(f(xd, pd), (xd, pd))
    g = torch.Generator(device=DEV).manual_seed(1)
    dx, dp = (torch.randn(v.shape, generator=g, device=DEV, dtype=torch.float64) for v in (xd, pd))
    with torch.no_grad():
        step = 2.0 ** -17                     # its square is 2^-34: third-order terms; rounding 2^-52 / 2^-17 = 2^-35
        slope = (f(xd + step * dx, pd + step * dp) - f(xd - step * dx, pd - step * dp)) / (2 * step)
        parts = [(ref[0] * dx).sum(), (ref[1] * dp).sum()]
        size = (ref[0] * dx).abs().sum() + (ref[1] * dp).abs().sum()
        assert float((slope - sum(parts)).abs() / size) < 2.0 ** -24
        for a, r in zip(got, ref):
            assert float((a.double() - r).norm() / r.norm()) <= 6 * 2.0 ** -8
        assert got[1][0, 1] == 0 and got[1][T - 1, 0] == 0   # slots that set nothing


@gpu
@pytest.mark.parametrize("wanted", ["", "W1", "W2"])
def test_frozen_bf16_weights(moe, wanted):
    """The gradients that are asked for do not change with those that are not; CTA pairs and single CTAs."""
    for E, I, T in ((8, 256, 40), (32, 768, 700)):
        g = torch.Generator(device=DEV).manual_seed(E)
        rnd = lambda *s: (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).bfloat16()  # noqa: E731
        t = dict(x=rnd(T, 512), W1=rnd(E, 2 * I, 512), W2=rnd(E, 512, I), p=torch.rand(T, 2, generator=g, device=DEV))
        idx = torch.rand(T, E, generator=g, device=DEV).topk(2, dim=1).indices
        grad = rnd(T, 512)

        def run(names):
            leaf = {k: v.detach().requires_grad_(k in names) for k, v in t.items()}
            out = moe.moe_layer(leaf["x"], idx, leaf["p"], leaf["W1"], leaf["W2"], 64)
            return dict(zip(names, torch.autograd.grad(out, [leaf[k] for k in names], grad)))

        whole = run(["x", "p", "W1", "W2"])
        for k, v in run(["x", "p", *wanted.split()]).items():
            assert torch.equal(v, whole[k]), k


@gpu
def test_memory_through_codes(moe):
    """A layer that waits for its backward holds codes, not weights as values."""
    T, H, E, K, I = 16, 1024, 64, 2, 512
    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    (q1, s1), (q2, s2) = moe.moe_quantize_fp4_block(rnd(E, 2 * I, H)), moe.moe_quantize_fp4_block(rnd(E, H, I))
    x, p = rnd(T, H).requires_grad_(), torch.rand(T, K, generator=g, device=DEV)
    idx = torch.rand(T, E, generator=g, device=DEV).topk(K, dim=1).indices
    bf16 = 2 * (E * 2 * I * H + E * H * I)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    out = moe.moe_layer_fp4_block(x, idx, p, q1, s1, q2, s2)
    assert torch.cuda.memory_allocated() - before < bf16 // 16
    torch.cuda.reset_peak_memory_stats()
    torch.autograd.grad(out, x, torch.ones_like(out))
    assert torch.cuda.max_memory_allocated() - before < bf16 + bf16 // 16    # the values once, no gradients of them


@gpu
def test_opcheck(moe):
    x, idx, p, W1, W2, grad = _case(moe, 6)
    W1, W2 = W1.bfloat16(), W2.bfloat16()
    ns = torch.ops.moe_gb300
    rmap, probs, _, status = ns.route_to_multihot(idx, p, 8)
    xd, *lay = ns.dispatch(x, rmap, probs, status, 3, 1)
    _, h, o, gu = ns.grouped_experts(xd, W1, W2, lay, 6, 3, 1, True)
    g_o, _ = ns.combine_backward(grad, o, lay, 6, 3, 1, 8)
    # (no comparison of outputs, as for experts_backward: rows behind the last expert's are not written)
    torch.library.opcheck(ns.experts_backward_rows.default, (g_o, xd, h, gu, W1, W2, lay, 6, 3, 1),
                          test_utils=("test_schema", "test_autograd_registration", "test_faketensor"))
