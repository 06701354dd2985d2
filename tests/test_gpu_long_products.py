"""Products that last longer than the limit of a wait are whole: in a pair of CTAs the
odd one waits for the even one's last operations from start to end, and its limit
counts only while its own loads stand still.  (A product takes 2 s from about 1.3e16
operations in 4 bits; here the limit is shortened instead.)"""
import contextlib

import pytest
import torch

gpu = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_topk_multihot_gb300 as m
    return m


@contextlib.contextmanager
def _limit(moe, us):
    lib = moe._native.lib
    assert lib.moe_selftest_pair_wait(us * 1000) == 0
    try:
        yield
    finally:
        assert lib.moe_selftest_pair_wait(-1) == 0


def test_refusals_without_a_gpu(moe):
    N = moe._native
    for ns in (0, -2, 2 * 10 ** 9 + 1):
        assert N.lib.moe_selftest_pair_wait(ns) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_selftest_pair_wait(-1) == 0


# tiles of 256, 128 and 192 columns, for at least four times the limit; 256 also with rows that do not start on 16 bytes
@gpu
@pytest.mark.parametrize("M,N,K", [(8192, 8192, 8192), (8191, 8191, 8192), (256, 4096, 131072), (512, 7168, 131072)])
def test_matmul_fp4(moe, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + N)
    a, b = (moe.moe_quantize_fp4_block(torch.randn(n, K, generator=g, device=DEV)) for n in (M, N))
    whole = moe.moe_matmul_fp4_block(*a, *b)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    with _limit(moe, 30):
        out = moe.moe_matmul_fp4_block(*a, *b, status=status)
    assert int(status) == 0 and not whole.isnan().any() and torch.equal(out, whole)


# (called one by one: autograd would run the backward on a thread of its own, whose limit is the usual one)
@gpu
@pytest.mark.parametrize("backward", [False, True])
def test_grouped_products(moe, backward):
    """The grouped products, forward and backward, each of 0.5 ms or more; the limit is 0.25 ms (a tile of the weights'
    gradients takes 0.09)."""
    T, H, E, K, I = 65536, 2048, 32, 4, 768
    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).bfloat16()  # noqa: E731
    x, W1, W2, p = rnd(T, H), rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5), torch.rand(T, K, generator=g, device=DEV)
    idx = torch.rand(T, E, generator=g, device=DEV).topk(K, dim=1).indices
    f = moe.moe_layer_forward(x, idx, p, W1, W2, 64, host_sync=False, save_for_backward=True)
    if backward:
        g_o, _ = moe.moe_combine_backward(rnd(T, H), f.layout, o_save=f.o, scaled=True)
        run = lambda: moe.moe_grouped_experts_backward(g_o, f.x_disp, f.h, f.gu, f.layout, W1, W2, scaled=True)  # noqa: E731
    else:
        run = lambda: moe.moe_grouped_experts(f.x_disp, f.layout, W1, W2, save_o=True, save_gu=True).values()  # noqa: E731
    rows = f.layout.row_token >= 0                     # (others are not all written)
    cut = lambda out: [t[rows] if t.shape[0] == f.layout.capacity else t for t in out]  # noqa: E731
    whole = cut(run())
    torch.cuda.synchronize()
    assert int(f.layout.status) == 0 and all(t.isfinite().all() for t in whole)
    with _limit(moe, 250):
        got = cut(run())
        torch.cuda.synchronize()
    assert int(f.layout.status) == 0 and all(torch.equal(a, b) for a, b in zip(got, whole))
