"""The example serves from 4 bits what its codes stand for."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def test_serving_from_codes():
    """The batch goes through the bf16 experts on the codes' values, bit for bit; tokens one at a time through the layer for few
    tokens: both layers within 2^-7 by the norm of each block's output, the stream's sum of two blocks within 2^-6."""
    import combine_topk_multihot_gb300 as moe
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    make = lambda: ex.Stack(2, 512, 16, 4, 256)  # noqa: E731
    x = torch.randn(64, 512, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    off = ex.serve(make(), x)
    assert off["fp4"] > 0 and off["fp4 one"] < 2.0 ** -6 and off["fp8 one"] < 2.0 ** -6
    coded, plain = make(), make()
    coded.to_fp4()
    for b, ((q1, s1), (q2, s2)) in zip(plain.blocks, coded.fp4):
        b["W1"], b["W2"] = moe.moe_dequantize_fp4_block(q1, s1), moe.moe_dequantize_fp4_block(q2, s2)
    with torch.no_grad():
        want, bf16 = plain(x), make()(x)
        assert torch.equal(coded(x), want)
    assert off["fp4"] == float((want.float() - bf16.float()).norm() / bf16.float().norm())
