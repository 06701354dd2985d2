"""Sizes past 32 bits of the block-scaled e4m3 operators are refused, on the host."""
import ctypes

import pytest
import torch

import combine_topk_multihot_gb300 as moe
from combine_topk_multihot_gb300 import _native as N, block


def test_sizes_past_32_bits_are_refused_without_a_gpu(monkeypatch):
    """K above 2^31 - 128, which rounded up to whole blocks passes 32 bits, and sizes that would lose their upper bits."""
    p = ctypes.c_void_p(256)
    for K in (2 ** 31 - 128, 2 ** 31 - 112, 2 ** 31 - 16):
        for M in (1, 9):
            assert N.lib.moe_matmul_fp8_block(p, p, M, p, p, 8, K, p, None, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
            assert b"2^31 - 256" in N.lib.moe_last_error()
    monkeypatch.setattr(block, "_on_gpu", lambda t, name: t.device)
    big = lambda *s, dt=torch.uint8: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="below 2\\^31"):
        moe.moe_quantize_fp8_block(big(1, 2 ** 32 + 16, dt=torch.bfloat16))
    small, scales = big(8, 16), big(8, 1, dt=torch.float32)
    for a, b in ((big(1, 2 ** 32 + 16), small), (big(2 ** 32 + 1, 16), small), (small, big(2 ** 32 + 1, 16))):
        with pytest.raises(ValueError, match="below 2\\^31"):
            moe.moe_matmul_fp8_block(a, scales, b, scales)
