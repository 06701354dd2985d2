"""The operators around the layer as custom operators: autograd through a whole
block against fp64 autograd of the formulas, opcheck, and the example that
trains and serves a stack of blocks."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_multihot_gb300 as m
    return m


def _rms(v, w):
    return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w


@pytest.mark.parametrize("use", ["both", "stream", "next"])
@pytest.mark.parametrize("gate_shape", ["token", "element", "none"])
def test_norm_autograd(moe, use, gate_shape):
    """Gradients of a loss of the stream, of the next norm, or of both.  fp32
    tensors, so that only y, next and their gradients (bf16) round: a gradient's
    random elements are off by 2^-9 of themselves at the most, 0.004 in the
    2-norm; the oracle's own bf16 roundings of next and of its gradient do the
    same, so 0.012 in all."""
    g = torch.Generator().manual_seed(3)
    T, H = 50, 320
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    x, y, w, w2 = rnd(T, H), rnd(T, H).bfloat16(), rnd(H), rnd(H)
    gate = {"token": rnd(T), "element": rnd(T, H), "none": None}[gate_shape]
    a, b = rnd(T, H), rnd(T, H).bfloat16()
    args = [t.clone().requires_grad_(True) if t is not None else None for t in (x, y, w, gate, w2)]
    out, nxt, _, _ = torch.ops.moe_gb300.norm_out(args[0], args[1], args[2], args[3], args[4], 0.5, True, 1e-6, 0.0)
    loss = (out * a).sum() * (use != "next") + (nxt.float() * b.float()).sum() * (use != "stream")
    if use == "next":
        loss = (nxt.float() * b.float()).sum()
    if use == "stream":
        loss = (out * a).sum()
    used = [t for i, t in enumerate(args) if t is not None and not (use == "stream" and i == 4)]
    grads = torch.autograd.grad(loss, used)
    ref = [t.detach().double().requires_grad_(True) for t in used]
    it = iter(ref)
    rx, ry, rw = next(it), next(it), next(it)
    rg = next(it) if gate is not None else None
    s = 1.0 if rg is None else torch.sigmoid(rg)[:, None] if gate_shape == "token" else torch.sigmoid(rg)
    ro = 0.5 * rx + s * _rms(ry, rw)
    rl = 0.0
    if use != "next":
        rl = rl + (ro * a.double()).sum()
    if use != "stream":
        rl = rl + (_rms(ro, next(it)) * b.double()).sum()
    for got, want in zip(grads, torch.autograd.grad(rl, ref)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 0.012, rel


def test_opcheck(moe):
    """Schemas, fake implementations and autograd registration."""
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    x, y, w, gate = rnd(9, 256).bfloat16(), rnd(9, 256).bfloat16(), rnd(256), rnd(9)
    ns = torch.ops.moe_gb300
    tests = ("test_schema", "test_autograd_registration", "test_faketensor")
    torch.library.opcheck(ns.norm_in.default, (x.requires_grad_(), w.requires_grad_(), 1e-6, 0.0), test_utils=tests)
    for gt in (None, gate):
        for w2 in (None, w.detach()):
            torch.library.opcheck(ns.norm_out.default, (x, y, w, gt, w2, 0.5, True, 1e-6, 0.0), test_utils=tests)
    codes, scales = ns.quantize_fp8_block(y, 1)
    torch.library.opcheck(ns.quantize_fp8_block.default, (y, 128), test_utils=tests)
    bq, bs = ns.quantize_fp8_block(rnd(40, 256).bfloat16(), 128)
    torch.library.opcheck(ns.matmul_fp8_block.default, (codes, scales, bq, bs), test_utils=tests)


def test_layer_fp8_block_is_its_steps(moe):
    """moe_layer_fp8_block = multihot, dispatch, experts, combine, and near the bf16 layer."""
    from tests._util import random_routing
    T, H, E, K, I = 70, 512, 8, 2, 256
    g = torch.Generator().manual_seed(5)
    idx, p = random_routing(T, E, K, seed=5)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    W1, W2 = ((torch.randn(E, *s, generator=g) * 0.05).bfloat16().to(DEV) for s in ((2 * I, H), (H, I)))
    (q1, s1), (q2, s2) = moe.moe_quantize_fp8_block(W1, 128), moe.moe_quantize_fp8_block(W2, 128)
    out = moe.moe_layer_fp8_block(x, idx.to(DEV), p.to(DEV), q1, s1, q2, s2)
    L = moe.Layout(T, E, K, 1, T * K, device=DEV)
    xd, _, _ = moe.moe_dispatch_topk(x, idx.to(DEV), p.to(DEV), L, host_sync=False)
    assert torch.equal(out, moe.moe_combine(moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2), L))
    ref = moe.moe_layer(x, idx.to(DEV), p.to(DEV), W1, W2)
    # four e4m3 roundings (x, W1, h, W2) of at most 2^-4 each, uniform: 2^-4 / sqrt(3) / sqrt(2) each at the most
    assert float((out.float() - ref.float()).norm() / ref.float().norm()) <= 4 ** 0.5 * 2.0 ** -4 / 6 ** 0.5 * 1.5


@pytest.mark.parametrize("bits", ["8", "32"])
def test_example(moe, bits):
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, fp8, one = ex.main(["--state-bits", bits, "--steps", "12"])
    assert all(b < a for a, b in zip(losses, losses[4:])) and losses[-1] < 0.9 * losses[0]
    assert fp8 < 0.05 and one < 0.02


def test_fp8_block_status(moe):
    """An expert index out of range, and a wait that runs out, reach the caller
    of the inference layer through its status."""
    T, H, E, K, I = 16, 256, 4, 2, 128
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    q1, s1 = moe.moe_quantize_fp8_block(torch.randn(E, 2 * I, H, generator=g).bfloat16().to(DEV), 128)
    q2, s2 = moe.moe_quantize_fp8_block(torch.randn(E, H, I, generator=g).bfloat16().to(DEV), 128)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(DEV)
    p = torch.rand(T, K, generator=g).to(DEV)
    call = lambda: moe.moe_layer_fp8_block(x, idx, p, q1, s1, q2, s2, return_status=True)  # noqa: E731
    out, status = call()
    assert int(status) == 0 and torch.equal(out, moe.moe_layer_fp8_block(x, idx, p, q1, s1, q2, s2))
    idx[3, 1] = E
    assert int(call()[1]) == 1
    idx[3, 1] = -1
    try:
        moe._native.lib.moe_selftest_block_product_tiles(0)
        out, status = call()
    finally:
        moe._native.lib.moe_selftest_block_product_tiles(-1)
    assert int(status) == moe._native.MOE_DEVERR_TIMEOUT and out.isnan().all()


def test_opcheck_dynamic(moe):
    """The operators under AOT dispatch with symbolic sizes, gradients among them."""
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    ns, tests = torch.ops.moe_gb300, ("test_aot_dispatch_dynamic",)
    x, y, w = rnd(9, 256).bfloat16().requires_grad_(), rnd(9, 256).bfloat16().requires_grad_(), rnd(256).requires_grad_()
    torch.library.opcheck(ns.norm_in.default, (x, w, 1e-6, 0.0), test_utils=tests)
    for gate in (None, rnd(9).requires_grad_(), rnd(9, 256).requires_grad_()):
        for w2 in (None, rnd(256).requires_grad_()):
            torch.library.opcheck(ns.norm_out.default, (x, y, w, gate, w2, 0.5, True, 1e-6, 0.0), test_utils=tests)
    codes, scales = ns.quantize_fp8_block(y.detach(), 1)
    torch.library.opcheck(ns.quantize_fp8_block.default, (y.detach(), 128), test_utils=tests)
    bq, bs = ns.quantize_fp8_block(rnd(40, 256).bfloat16(), 128)
    torch.library.opcheck(ns.matmul_fp8_block.default, (codes, scales, bq, bs), test_utils=tests)
