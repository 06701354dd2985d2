"""A block-scaled product whose operands stop arriving ends by its own bounded
waits (about 2 s), says so in the status word, and leaves NaN wherever it did
not get to: it cannot pass for a finished one."""
import contextlib

import pytest
import torch

from tests._util import random_routing

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_multihot_gb300 as m
    return m


@contextlib.contextmanager
def _tiles(moe, n):
    lib = moe._native.lib
    assert lib.moe_selftest_block_product_tiles(n) == moe._native.MOE_OK
    try:
        yield
    finally:
        assert lib.moe_selftest_block_product_tiles(-1) == moe._native.MOE_OK


# tiles of 64, 128 and 256 columns, no tile reached; then several tiles a CTA of
# which the first is done, with rows that start on 16 bytes and rows that do not
@pytest.mark.parametrize("M,N,K,tiles", [(100, 513, 512, 0), (1000, 4096, 384, 0), (2049, 4096, 256, 0), (5000, 8192, 384, 1),
                                         (5001, 8195, 384, 1)])
def test_matmul(moe, M, N, K, tiles):
    g = torch.Generator().manual_seed(M)
    aq, sa = moe.moe_quantize_fp8_block(torch.randn(M, K, generator=g).bfloat16().to(DEV))
    bq, sb = moe.moe_quantize_fp8_block(torch.randn(N, K, generator=g).bfloat16().to(DEV), 128)
    whole = moe.moe_matmul_fp8_block(aq, sa, bq, sb)
    for status in (None, torch.zeros(1, dtype=torch.int32, device=DEV)):
        out = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
        with _tiles(moe, tiles):
            moe.moe_matmul_fp8_block(aq, sa, bq, sb, out=out, status=status)
        torch.cuda.synchronize()
        missing = out.isnan()
        assert missing.all() if tiles == 0 else missing.any() and not missing.all()
        assert torch.equal(out[~missing], whole[~missing])
        if status is not None:
            assert int(status) == moe._native.MOE_DEVERR_TIMEOUT
    assert torch.equal(moe.moe_matmul_fp8_block(aq, sa, bq, sb), whole)


def test_experts(moe):
    T, H, E, K, I = 900, 512, 8, 2, 256
    g = torch.Generator().manual_seed(1)
    idx, p = random_routing(T, E, K, seed=1)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    q1, s1 = moe.moe_quantize_fp8_block((torch.randn(E, 2 * I, H, generator=g) * 0.05).bfloat16().to(DEV), 128)
    q2, s2 = moe.moe_quantize_fp8_block((torch.randn(E, H, I, generator=g) * 0.05).bfloat16().to(DEV), 128)
    L = moe.Layout(T, E, K, 1, T * K, device=DEV)
    xd, _, _ = moe.moe_dispatch_topk(x, idx.to(DEV), p.to(DEV), L, host_sync=False)
    whole = moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2)
    with _tiles(moe, 0):
        y = moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2, out=torch.zeros_like(whole))
    torch.cuda.synchronize()
    assert y.isnan().all() and int(L.status) == moe._native.MOE_DEVERR_TIMEOUT
    L.status.zero_()
    assert torch.equal(moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2), whole) and int(L.status) == 0


def test_refuses(moe):
    assert moe._native.lib.moe_selftest_block_product_tiles(-2) == moe._native.MOE_ERR_INVALID_ARG
