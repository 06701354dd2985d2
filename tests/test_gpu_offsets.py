"""Slices of larger tensors: what a kernel reads value by value may start at
any element.  Each call on slices gives the bits of the call on copies."""
import pytest
import torch

from tests._util import random_routing

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_multihot_gb300 as m
    return m


def _off(t, by=1):
    """t's values in memory that starts `by` elements after an aligned address."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=t.device)
    flat[by:].copy_(t.reshape(-1))
    out = flat[by:].view(t.shape)
    assert out.data_ptr() % 16
    return out


def _same(a, b):
    for x, y in zip(a, b):
        assert (x is None and y is None) or torch.equal(x, y)


# rows of a multiple of 8 values: weights, statistics and gates per token; others: everything
@pytest.mark.parametrize("T,H", [(5, 256), (1300, 2048), (3, 33), (700, 1001), (2, 8193)])
@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_norms(moe, T, H, xt, wt):
    g = torch.Generator().manual_seed(H)
    rnd = lambda *s, dt=F32: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
    rows = _off if H % 8 else (lambda t: t)
    x, y, w, w2, gate = rnd(T, H, dt=xt), rnd(T, H, dt=BF16), rnd(H, dt=wt), rnd(H, dt=wt), rnd(T, dt=wt)
    first = moe.moe_norm_in(x, w, save_rstd=True)
    _same(first, moe.moe_norm_in(rows(x), _off(w), save_rstd=True))
    dn = rnd(T, H, dt=BF16)
    _same(moe.moe_norm_in_backward(dn, x, w, first[1], grad_res=x),
          moe.moe_norm_in_backward(rows(dn), rows(x), _off(w), _off(first[1]), grad_res=rows(x)))
    fwd = moe.moe_norm_out(x, y, w, gate=gate, next_weight=w2, save_rstd=True)
    _same(fwd, moe.moe_norm_out(rows(x), rows(y), _off(w), gate=_off(gate), next_weight=_off(w2), save_rstd=True))
    out, rstd, _, rstd2 = fwd
    _same(moe.moe_norm_out_backward(x, y, w, rstd, gate=gate, grad_next=dn, out=out, next_weight=w2, next_rstd=rstd2),
          moe.moe_norm_out_backward(rows(x), rows(y), _off(w), _off(rstd), gate=_off(gate), grad_next=rows(dn), out=rows(out),
                                    next_weight=_off(w2), next_rstd=_off(rstd2)))
    element = rnd(T, H, dt=BF16)
    _same(moe.moe_norm_out_backward(x, y, w, rstd, gate=element),
          moe.moe_norm_out_backward(rows(x), rows(y), _off(w), _off(rstd), gate=rows(element)))


def test_weights_on_another_stream(moe):
    """Weights that have to be copied are copied on the stream of the call."""
    x, w = torch.randn(64, 512, device=DEV), _off(torch.zeros(512, device=DEV))
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            a = torch.tanh(a @ a)
        w.add_(1.0)
    n, _ = moe.moe_norm_in(x, w, stream=side)
    side.synchronize()
    assert torch.equal(n, moe.moe_norm_in(x, torch.ones(512, device=DEV))[0])


def test_operators_take_slices(moe):
    """A chunk of a batch of odd rows, and a gate of its tokens, as a program that works through chunks has them."""
    T, H = 9, 321
    g = torch.Generator().manual_seed(2)
    x, y = torch.randn(T, H, generator=g).bfloat16().to(DEV), torch.randn(T, H, generator=g).bfloat16().to(DEV)
    w, gate = torch.ones(H, device=DEV), torch.randn(T, generator=g).to(DEV)
    whole = torch.ops.moe_gb300.norm_out(x, y, w, gate, w, 0.5, True, 1e-6, 0.0)
    part = torch.ops.moe_gb300.norm_out(x[1:], y[1:], w, gate[1:], w, 0.5, True, 1e-6, 0.0)
    _same([t[1:] for t in whole], part)


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("N", [256, 129])
def test_scales(moe, M, N):
    K = 384
    g = torch.Generator().manual_seed(M + N)
    a, sa = moe.moe_quantize_fp8_block(torch.randn(M + 1, K, generator=g).bfloat16().to(DEV))
    b, sb = moe.moe_quantize_fp8_block(torch.randn(N, K, generator=g).bfloat16().to(DEV), 128)
    assert sa[1:].data_ptr() % 16
    out = _off(torch.zeros(M, N, dtype=BF16, device=DEV)) if N % 8 else None
    got = moe.moe_matmul_fp8_block(a[1:], sa[1:], b, _off(sb), out=out)
    assert torch.equal(got, moe.moe_matmul_fp8_block(a[1:].clone(), sa[1:].clone(), b, sb))
    src = torch.randn(N, K, generator=g).bfloat16().to(DEV)
    for block_rows in (1, 128):
        codes, scales = moe.moe_quantize_fp8_block(src, block_rows)
        _same((codes, scales), moe.moe_quantize_fp8_block(src, block_rows, out=(torch.zeros_like(codes), _off(torch.zeros_like(scales)))))


@pytest.mark.parametrize("T", [4, 40])
def test_expert_scales(moe, T):
    H, E, K, I = 256, 4, 2, 128
    g = torch.Generator().manual_seed(T)
    idx, p = random_routing(T, E, K, seed=T)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    q1, s1 = moe.moe_quantize_fp8_block(torch.randn(E, 2 * I, H, generator=g).bfloat16().to(DEV), 128)
    q2, s2 = moe.moe_quantize_fp8_block(torch.randn(E, H, I, generator=g).bfloat16().to(DEV), 128)
    L = moe.Layout(T, E, K, 1, T * K, device=DEV)
    xd, _, _ = moe.moe_dispatch_topk(x, idx.to(DEV), p.to(DEV), L, host_sync=False)
    assert torch.equal(moe.moe_grouped_experts_fp8_block(xd, L, q1, _off(s1), q2, _off(s2)),
                       moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2))
