"""Tensors or a stream on a device other than the current one are refused
before anything is launched.  One device is enough: another is only claimed to
be the current one."""
import types

import pytest
import torch

import combine_topk_multihot_gb300 as moe
from combine_topk_multihot_gb300 import block, moe as core


def _elsewhere(monkeypatch, current):
    monkeypatch.setattr(core, "_current_device", lambda: current)


def test_refused_without_a_gpu(monkeypatch):
    _elsewhere(monkeypatch, 0)
    monkeypatch.setattr(block, "_current_raw_stream", lambda index: 77 + index)
    there = types.SimpleNamespace(is_cuda=True, get_device=lambda: 1, is_contiguous=lambda: True, data_ptr=lambda: 256,
                                  numel=lambda: 4)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        core._ptr(there)
    other = types.SimpleNamespace(device_index=1, cuda_stream=0)     # a default stream's handle is 0 on any device
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        core._stream(other)
    with pytest.raises(ValueError, match="tensors are on cuda:1"):
        block._raw_stream(None, torch.device("cuda:1"))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        block._raw_stream(other, torch.device("cuda:0"))
    assert block._raw_stream(None, torch.device("cuda:0")) == 77
    assert core._ptr(torch.zeros(3)).value        # host memory (of the oracle's own calls) is not on a device


@pytest.mark.gpu
def test_every_call_refuses(monkeypatch):
    dev, T, H, E, K, I = "cuda", 4, 256, 8, 2, 128
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    x, w, r = bf(T, H), torch.ones(H, device=dev), torch.ones(T, device=dev)
    codes, scales = moe.moe_quantize_fp8_block(x)
    wq, ws = moe.moe_quantize_fp8_block(bf(128, H), 128)
    q1, s1 = moe.moe_quantize_fp8_block(bf(E, 2 * I, H), 128)
    q2, s2 = moe.moe_quantize_fp8_block(bf(E, H, I), 128)
    L = moe.Layout(T, E, K, 1, T * K, device=dev)
    opt = moe.AdamWState([w])
    logits = torch.zeros(T, E, device=dev)
    calls = [lambda: moe.moe_norm_in(x, w), lambda: moe.moe_norm_in_backward(x, x, w, r), lambda: moe.moe_norm_out(x, x, w),
             lambda: moe.moe_norm_out_backward(x, x, w, r), lambda: moe.moe_adamw_step(opt, [w], 1e-3),
             lambda: moe.moe_quantize_fp8_block(x), lambda: moe.moe_matmul_fp8_block(codes, scales, wq, ws),
             lambda: moe.moe_grouped_experts_fp8_block(bf(T * K, H), L, q1, s1, q2, s2),
             lambda: moe.moe_router_topk(logits, K), lambda: moe.moe_combine(bf(T * K, H), L),
             lambda: torch.ops.moe_gb300.norm_in(x, w, 1e-6, 0.0)]
    _elsewhere(monkeypatch, torch.cuda.current_device() + 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    assert opt.step == 0
