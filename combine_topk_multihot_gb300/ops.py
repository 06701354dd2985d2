"""The MoE layer as PyTorch custom operators, with autograd.

Page cited: "Add the deepep expert-parallel implementation
(huggingface/transformers #49638)", What this adds, Custom ops.  There the
dispatch, the combine and the combine's backward become torch.library
operators, each with a shape-only ("fake") implementation for tracing and an
autograd rule, and the dispatch handle, which no operator can carry, travels
between them as its component tensors and is put back together on the far
side.  Here every step of the layer is such an operator: the router (with
its gradient registered on the operator), multihot, dispatch, grouped
experts, combine, and the four backward steps.  So are the norms before and
after a block (norm_in and norm_out, with their gradients) and the block-scaled
e4m3 quantiser, product and experts.

Every operator takes the sync-free route: the expanded buffers are sized for
the worst case (T*K + E*(pad_multiple - 1) rows), nothing is read back to the
host, and each output's shape is a function of the input shapes alone -- so the
layer can be captured in a CUDA graph and traced by torch.compile with
fullgraph=True.  The operators are registered for CUDA only (a CPU tensor gets
PyTorch's "no kernel" error) and only marshal arguments to the C library; all
arithmetic runs in its CUDA kernels.
"""
from __future__ import annotations

from typing import List, Optional, Tuple

import torch
from torch import Tensor

from . import block as _b
from . import moe as _m

NS = "moe_gb300"


def _capacity(T, E, K, P):
    return T * K + E * (P - 1)


def _layout(T: int, E: int, K: int, P: int, lay: List[Tensor]) -> _m.Layout:
    return _m.Layout.from_tensors(T, E, K, P, lay)


def _layout_fake(T, E, K, P, device) -> Tuple[Tensor, ...]:
    """Shapes and dtypes of Layout.tensors()."""
    C = _capacity(T, E, K, P)
    i32 = dict(dtype=torch.int32, device=device)
    return (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(2, **i32),
            torch.empty(C, **i32), torch.empty(C, **i32),
            torch.empty(C, dtype=torch.float32, device=device), torch.empty(T * K, **i32),
            torch.empty(1, **i32))


# ------------------------------------------------------------------ router
@torch.library.custom_op(f"{NS}::router_topk", mutates_args=(), device_types="cuda")
def router_topk(logits: Tensor, top_k: int) -> Tuple[Tensor, Tensor]:
    """(topk_idx int64 [T, K], topk_probs fp32 [T, K]): softmax, top-k, renormalise."""
    return _m.moe_router_topk(logits.contiguous(), top_k)


@router_topk.register_fake
def _(logits, top_k):
    T = logits.shape[0]
    return (torch.empty(T, top_k, dtype=torch.int64, device=logits.device),
            torch.empty(T, top_k, dtype=torch.float32, device=logits.device))


@torch.library.custom_op(f"{NS}::router_topk_backward", mutates_args=(), device_types="cuda")
def router_topk_backward(grad_topk_probs: Tensor, topk_probs: Tensor, topk_idx: Tensor,
                         num_experts: int) -> Tensor:
    """grad_logits fp32 [T, E]."""
    return _m.moe_router_topk_backward(grad_topk_probs.contiguous(), topk_probs, topk_idx, num_experts)


@router_topk_backward.register_fake
def _(grad_topk_probs, topk_probs, topk_idx, num_experts):
    return torch.empty(topk_idx.shape[0], num_experts, dtype=torch.float32, device=topk_idx.device)


def _router_setup(ctx, inputs, output):
    logits, _ = inputs
    idx, w = output
    ctx.save_for_backward(idx, w)
    ctx.num_experts = logits.shape[1]
    ctx.mark_non_differentiable(idx)


def _router_backward(ctx, grad_idx, grad_w):
    idx, w = ctx.saved_tensors
    if grad_w is None:
        return None, None
    return torch.ops.moe_gb300.router_topk_backward(grad_w, w, idx, ctx.num_experts), None


torch.library.register_autograd(f"{NS}::router_topk", _router_backward, setup_context=_router_setup)


# ------------------------------------------------------------------ forward
@torch.library.custom_op(f"{NS}::route_to_multihot", mutates_args=(), device_types="cuda")
def route_to_multihot(topk_idx: Tensor, topk_probs: Tensor,
                      num_experts: int) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    """(routing_map uint8 [T, E], probs fp32 [T, E], winner_slot int8 [T, E], status int32 [1])."""
    status = torch.zeros(1, dtype=torch.int32, device=topk_idx.device)
    rmap, probs, win = _m.moe_route_to_multihot(topk_idx.contiguous(), topk_probs.contiguous(),
                                                num_experts, status)
    return rmap, probs, win, status


@route_to_multihot.register_fake
def _(topk_idx, topk_probs, num_experts):
    T, d = topk_idx.shape[0], topk_idx.device
    return (torch.empty(T, num_experts, dtype=torch.uint8, device=d),
            torch.empty(T, num_experts, dtype=torch.float32, device=d),
            torch.empty(T, num_experts, dtype=torch.int8, device=d),
            torch.empty(1, dtype=torch.int32, device=d))


@torch.library.custom_op(f"{NS}::dispatch", mutates_args=(), device_types="cuda")
def dispatch(x: Tensor, routing_map: Tensor, probs: Tensor, status: Tensor, top_k: int,
             pad_multiple: int) -> Tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor, Tensor,
                                         Tensor, Tensor]:
    """Sync-free dispatch: (x_disp [C, H], *Layout.tensors()).  ``status``
    carries the multihot step's device error bits; the layout gets a copy."""
    T, H = x.shape
    E = routing_map.shape[1]
    lay = _m.Layout(T, E, top_k, pad_multiple, _capacity(T, E, top_k, pad_multiple),
                    device=x.device, status=status.clone())
    x_disp, _ = _m.moe_dispatch(x.contiguous(), routing_map, probs, lay, host_sync=False)
    return (x_disp,) + lay.tensors()


@dispatch.register_fake
def _(x, routing_map, probs, status, top_k, pad_multiple):
    T, H = x.shape
    E = routing_map.shape[1]
    C = _capacity(T, E, top_k, pad_multiple)
    return (x.new_empty(C, H),) + _layout_fake(T, E, top_k, pad_multiple, x.device)


@torch.library.custom_op(f"{NS}::grouped_experts", mutates_args=(), device_types="cuda")
def grouped_experts(x_disp: Tensor, W1: Tensor, W2: Tensor, lay: List[Tensor], T: int, top_k: int,
                    pad_multiple: int, save_for_backward: bool) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    """(y [C, H], h [C, I], o [C, H], gu [C, 2I]); o and gu have no rows unless saving."""
    L = _layout(T, W1.shape[0], top_k, pad_multiple, lay)
    r = _m.moe_grouped_experts(x_disp, L, W1.contiguous(), W2.contiguous(), save_o=save_for_backward,
                               save_gu=save_for_backward)
    if save_for_backward:
        return r["y"], r["h"], r["o"], r["gu"]
    return r["y"], r["h"], x_disp.new_empty(0, x_disp.shape[1]), x_disp.new_empty(0, W1.shape[1])


@grouped_experts.register_fake
def _(x_disp, W1, W2, lay, T, top_k, pad_multiple, save_for_backward):
    C, H = x_disp.shape
    twoI = W1.shape[1]
    S = C if save_for_backward else 0
    return x_disp.new_empty(C, H), x_disp.new_empty(C, twoI // 2), x_disp.new_empty(S, H), \
        x_disp.new_empty(S, twoI)


@torch.library.custom_op(f"{NS}::combine", mutates_args=(), device_types="cuda")
def combine(y: Tensor, lay: List[Tensor], T: int, top_k: int, pad_multiple: int,
            num_experts: int) -> Tensor:
    """out [T, H]: the sum of each token's expert rows."""
    return _m.moe_combine(y, _layout(T, num_experts, top_k, pad_multiple, lay))


@combine.register_fake
def _(y, lay, T, top_k, pad_multiple, num_experts):
    return y.new_empty(T, y.shape[1])


# ------------------------------------------------------------------ backward
@torch.library.custom_op(f"{NS}::combine_backward", mutates_args=(), device_types="cuda")
def combine_backward(grad_out: Tensor, o_save: Tensor, lay: List[Tensor], T: int, top_k: int,
                     pad_multiple: int, num_experts: int) -> Tuple[Tensor, Tensor]:
    """(G_o [C, H], grad_w fp32 [C]): grad_out sent along the forward's layout
    with each row's routing weight applied (G_o = w * grad_y, the gradient of
    the experts' pre-weight output), and each row's routing-weight gradient."""
    L = _layout(T, num_experts, top_k, pad_multiple, lay)
    return _m.moe_combine_backward(grad_out.contiguous(), L, o_save=o_save, scaled=True)


@combine_backward.register_fake
def _(grad_out, o_save, lay, T, top_k, pad_multiple, num_experts):
    C = lay[3].shape[0]
    return grad_out.new_empty(C, grad_out.shape[1]), \
        torch.empty(C, dtype=torch.float32, device=grad_out.device)


@torch.library.custom_op(f"{NS}::experts_backward", mutates_args=(), device_types="cuda")
def experts_backward(g_o: Tensor, x_disp: Tensor, h: Tensor, gu_save: Tensor, W1: Tensor,
                     W2: Tensor, lay: List[Tensor], T: int, top_k: int,
                     pad_multiple: int) -> Tuple[Tensor, Tensor, Tensor]:
    """(grad_x_disp [C, H] bf16, dW1 fp32 [E, 2I, H], dW2 fp32 [E, H, I]) from
    combine_backward's G_o."""
    L = _layout(T, W1.shape[0], top_k, pad_multiple, lay)
    return _m.moe_grouped_experts_backward(g_o, x_disp, h, gu_save, L, W1.contiguous(),
                                           W2.contiguous(), scaled=True)


@experts_backward.register_fake
def _(g_o, x_disp, h, gu_save, W1, W2, lay, T, top_k, pad_multiple):
    return (x_disp.new_empty(x_disp.shape),
            torch.empty(W1.shape, dtype=torch.float32, device=W1.device),
            torch.empty(W2.shape, dtype=torch.float32, device=W2.device))


@torch.library.custom_op(f"{NS}::dispatch_backward", mutates_args=(), device_types="cuda")
def dispatch_backward(grad_x_disp: Tensor, grad_w: Tensor, lay: List[Tensor], T: int, top_k: int,
                      pad_multiple: int, num_experts: int) -> Tuple[Tensor, Tensor]:
    """(grad_x [T, H], grad_probs fp32 [T, E])."""
    L = _layout(T, num_experts, top_k, pad_multiple, lay)
    return _m.moe_dispatch_backward(grad_x_disp, L, grad_w=grad_w)


@dispatch_backward.register_fake
def _(grad_x_disp, grad_w, lay, T, top_k, pad_multiple, num_experts):
    return (grad_x_disp.new_empty(T, grad_x_disp.shape[1]),
            torch.empty(T, num_experts, dtype=torch.float32, device=grad_x_disp.device))


@torch.library.custom_op(f"{NS}::route_to_multihot_backward", mutates_args=(), device_types="cuda")
def route_to_multihot_backward(grad_probs: Tensor, topk_idx: Tensor, winner_slot: Tensor) -> Tensor:
    """grad_topk_probs fp32 [T, K]."""
    return _m.moe_route_to_multihot_backward(grad_probs.contiguous(), topk_idx.contiguous(),
                                             winner_slot)


@route_to_multihot_backward.register_fake
def _(grad_probs, topk_idx, winner_slot):
    return torch.empty(topk_idx.shape, dtype=torch.float32, device=topk_idx.device)


# ------------------------------------------------------------------ the layer
_ops = torch.ops.moe_gb300


class MoELayerFunction(torch.autograd.Function):
    """out = combine(experts(dispatch(x, multihot(topk_idx, topk_probs)), W1, W2)).

    The backward gives gradients for x, topk_probs, W1 and W2.  The kernels
    accumulate the weight gradients in fp32; autograd wants them in the
    weights' own dtype, so they are cast on the way out."""

    @staticmethod
    def forward(ctx, x, topk_idx, topk_probs, W1, W2, pad_multiple: int):
        T, K = topk_idx.shape
        E = W1.shape[0]
        rmap, probs, win, status = _ops.route_to_multihot(topk_idx, topk_probs, E)
        x_disp, *lay = _ops.dispatch(x, rmap, probs, status, K, pad_multiple)
        y, h, o, gu = _ops.grouped_experts(x_disp, W1, W2, lay, T, K, pad_multiple, True)
        out = _ops.combine(y, lay, T, K, pad_multiple, E)
        ctx.save_for_backward(topk_idx, win, x_disp, h, o, gu, W1, W2, *lay)
        ctx.meta = (T, K, E, pad_multiple)
        status = lay[-1]
        ctx.mark_non_differentiable(status)
        ctx.set_materialize_grads(False)   # no zero gradient is made for status
        return out, status

    @staticmethod
    def backward(ctx, grad_out, _grad_status):
        topk_idx, win, x_disp, h, o, gu, W1, W2, *lay = ctx.saved_tensors
        T, K, E, P = ctx.meta
        g_o, grad_w = _ops.combine_backward(grad_out, o, lay, T, K, P, E)
        gxd, dW1, dW2 = _ops.experts_backward(g_o, x_disp, h, gu, W1, W2, lay, T, K, P)
        grad_x, grad_probs = _ops.dispatch_backward(gxd, grad_w, lay, T, K, P, E)
        grad_topk = _ops.route_to_multihot_backward(grad_probs, topk_idx, win)
        return grad_x, None, grad_topk, dW1.to(W1.dtype), dW2.to(W2.dtype), None


def moe_layer(x: Tensor, topk_idx: Tensor, topk_probs: Tensor, W1: Tensor, W2: Tensor,
              pad_multiple: int = 1, return_status: bool = False):
    """The whole layer (a1..a6 forward, a7..a10 backward) as one differentiable
    call on the sync-free route.  Under torch.no_grad() the gate/up values and
    the pre-weight outputs are not saved.  With ``return_status`` it returns
    (out, status): status is the device's error word (MOE_DEVERR_* bits; 1 = an
    expert index outside [-1, E) was seen and dropped), left on the device so
    that reading it is the caller's choice of synchronisation point."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in (x, topk_probs, W1, W2)):
        out, status = MoELayerFunction.apply(x, topk_idx, topk_probs, W1, W2, pad_multiple)
    else:
        T, K = topk_idx.shape
        E = W1.shape[0]
        rmap, probs, win, status = _ops.route_to_multihot(topk_idx, topk_probs, E)
        x_disp, *lay = _ops.dispatch(x, rmap, probs, status, K, pad_multiple)
        y, h, o, gu = _ops.grouped_experts(x_disp, W1, W2, lay, T, K, pad_multiple, False)
        out = _ops.combine(y, lay, T, K, pad_multiple, E)
        status = lay[-1]
    return (out, status) if return_status else out


# ------------------------------------------------------------------ the norms around a block
@torch.library.custom_op(f"{NS}::norm_in", mutates_args=(), device_types="cuda")
def norm_in(x: Tensor, weight: Tensor, eps: float, weight_offset: float) -> Tuple[Tensor, Tensor]:
    """(norm bf16 [T, H], rstd fp32 [T])."""
    return _b.moe_norm_in(x.contiguous(), weight.contiguous(), eps, weight_offset, save_rstd=True)


@norm_in.register_fake
def _(x, weight, eps, weight_offset):
    return x.new_empty(x.shape, dtype=torch.bfloat16), x.new_empty(x.shape[0], dtype=torch.float32)


@torch.library.custom_op(f"{NS}::norm_in_backward", mutates_args=(), device_types="cuda")
def norm_in_backward(grad_norm: Tensor, x: Tensor, weight: Tensor, rstd: Tensor, weight_offset: float) -> Tuple[Tensor, Tensor]:
    """(grad_x, grad_weight fp32 [H])."""
    return _b.moe_norm_in_backward(grad_norm.contiguous(), x.contiguous(), weight.contiguous(), rstd,
                                   weight_offset=weight_offset)


@norm_in_backward.register_fake
def _(grad_norm, x, weight, rstd, weight_offset):
    return x.new_empty(x.shape), weight.new_empty(weight.shape, dtype=torch.float32)


def _norm_in_setup(ctx, inputs, output):
    x, weight, _, ctx.weight_offset = inputs
    ctx.save_for_backward(x, weight, output[1])
    ctx.mark_non_differentiable(output[1])
    ctx.set_materialize_grads(False)


def _norm_in_backward(ctx, grad_norm, _grad_rstd):
    x, weight, rstd = ctx.saved_tensors
    if grad_norm is None:
        return None, None, None, None
    gx, gw = torch.ops.moe_gb300.norm_in_backward(grad_norm, x, weight, rstd, ctx.weight_offset)
    return gx, gw.to(weight.dtype), None, None


torch.library.register_autograd(f"{NS}::norm_in", _norm_in_backward, setup_context=_norm_in_setup)


@torch.library.custom_op(f"{NS}::norm_out", mutates_args=(), device_types="cuda")
def norm_out(x: Tensor, y: Tensor, weight: Tensor, gate: Optional[Tensor], next_weight: Optional[Tensor],
             residual_scale: float, gate_sigmoid: bool, eps: float,
             weight_offset: float) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    """(out, next, rstd, next_rstd); next and next_rstd have no rows without a next norm."""
    out, rstd, nxt, next_rstd = _b.moe_norm_out(
        x.contiguous(), y.contiguous(), weight.contiguous(), None if gate is None else gate.contiguous(),
        residual_scale, gate_sigmoid, None if next_weight is None else next_weight.contiguous(), eps, weight_offset,
        save_rstd=True)
    if nxt is None:
        nxt, next_rstd = y.new_empty(0, x.shape[1]), rstd.new_empty(0)
    return out, nxt, rstd, next_rstd


@norm_out.register_fake
def _(x, y, weight, gate, next_weight, residual_scale, gate_sigmoid, eps, weight_offset):
    T, H = x.shape
    S = T if next_weight is not None else 0
    f32 = dict(dtype=torch.float32, device=x.device)
    return (x.new_empty(T, H), torch.empty(S, H, dtype=torch.bfloat16, device=x.device), torch.empty(T, **f32),
            torch.empty(S, **f32))


@torch.library.custom_op(f"{NS}::norm_out_backward", mutates_args=(), device_types="cuda")
def norm_out_backward(grad_out: Optional[Tensor], grad_next: Optional[Tensor], out: Optional[Tensor], y: Tensor,
                      weight: Tensor, gate: Optional[Tensor], rstd: Tensor, next_weight: Optional[Tensor],
                      next_rstd: Optional[Tensor], residual_scale: float, gate_sigmoid: bool,
                      weight_offset: float) -> Tuple[Tensor, Tensor, Tensor, Tensor, Tensor]:
    """(grad_x, grad_y, grad_gate, grad_weight fp32, grad_next_weight fp32); no elements where there is no such input."""
    opt = lambda t: None if t is None else t.contiguous()  # noqa: E731
    gx, gy, gg, gw, gw2 = _b.moe_norm_out_backward(
        opt(grad_out), y.contiguous(), weight.contiguous(), rstd, opt(gate), residual_scale, gate_sigmoid, opt(grad_next),
        opt(out), opt(next_weight), next_rstd, weight_offset)
    return gx, gy, rstd.new_empty(0) if gg is None else gg, gw, rstd.new_empty(0) if gw2 is None else gw2


@norm_out_backward.register_fake
def _(grad_out, grad_next, out, y, weight, gate, rstd, next_weight, next_rstd, residual_scale, gate_sigmoid, weight_offset):
    like = grad_out if grad_out is not None else out
    f32 = dict(dtype=torch.float32, device=y.device)
    return (like.new_empty(y.shape), y.new_empty(y.shape),
            torch.empty(0, **f32) if gate is None else gate.new_empty(gate.shape), torch.empty(weight.shape, **f32),
            torch.empty(weight.shape if next_weight is not None else 0, **f32))


def _norm_out_setup(ctx, inputs, output):
    x, y, weight, gate, next_weight, ctx.residual_scale, ctx.gate_sigmoid, _, ctx.weight_offset = inputs
    out, nxt, rstd, next_rstd = output
    ctx.save_for_backward(y, weight, gate, next_weight, rstd, out if next_weight is not None else None, next_rstd)
    ctx.mark_non_differentiable(*((rstd, next_rstd) if next_weight is not None else (nxt, rstd, next_rstd)))
    ctx.set_materialize_grads(False)
    ctx.x_dtype = x.dtype


def _norm_out_backward(ctx, grad_out, grad_next, _grad_rstd, _grad_next_rstd):
    y, weight, gate, next_weight, rstd, out, next_rstd = ctx.saved_tensors
    if grad_out is None and grad_next is None:
        return (None,) * 9
    if next_weight is None or grad_next is None:      # only the stream was used
        out = used = None
        if grad_out is None:
            return (None,) * 9
    else:
        used = next_weight
    gx, gy, gg, gw, gw2 = torch.ops.moe_gb300.norm_out_backward(
        grad_out, grad_next if used is not None else None, out, y, weight, gate, rstd, used,
        next_rstd if used is not None else None, ctx.residual_scale, ctx.gate_sigmoid, ctx.weight_offset)
    return (gx, gy, gw.to(weight.dtype), gg if gate is not None else None,
            gw2.to(used.dtype) if used is not None else None, None, None, None, None)


torch.library.register_autograd(f"{NS}::norm_out", _norm_out_backward, setup_context=_norm_out_setup)


# ------------------------------------------------------------------ block-scaled e4m3
@torch.library.custom_op(f"{NS}::quantize_fp8_block", mutates_args=(), device_types="cuda")
def quantize_fp8_block(src: Tensor, block_rows: int) -> Tuple[Tensor, Tensor]:
    """(codes uint8, scales fp32)."""
    return _b.moe_quantize_fp8_block(src.contiguous(), block_rows)


@quantize_fp8_block.register_fake
def _(src, block_rows):
    R, C = src.shape[-2:]
    return (src.new_empty(src.shape, dtype=torch.uint8),
            src.new_empty((*src.shape[:-2], (R + block_rows - 1) // block_rows, (C + 127) // 128), dtype=torch.float32))


@torch.library.custom_op(f"{NS}::matmul_fp8_block", mutates_args=(), device_types="cuda")
def matmul_fp8_block(a_q: Tensor, a_scale: Tensor, b_q: Tensor, b_scale: Tensor) -> Tensor:
    """a b^T, [M, N] bf16."""
    return _b.moe_matmul_fp8_block(a_q, a_scale, b_q, b_scale)


@matmul_fp8_block.register_fake
def _(a_q, a_scale, b_q, b_scale):
    return a_q.new_empty(a_q.shape[0], b_q.shape[0], dtype=torch.bfloat16)


@torch.library.custom_op(f"{NS}::grouped_experts_fp8_block", mutates_args=(), device_types="cuda")
def grouped_experts_fp8_block(x_disp: Tensor, W1_q: Tensor, W1_scale: Tensor, W2_q: Tensor, W2_scale: Tensor,
                              lay: List[Tensor], T: int, top_k: int, pad_multiple: int) -> Tensor:
    """y [C, H] bf16, for combine."""
    return _b.moe_grouped_experts_fp8_block(x_disp, _layout(T, W1_q.shape[0], top_k, pad_multiple, lay), W1_q, W1_scale,
                                            W2_q, W2_scale)


@grouped_experts_fp8_block.register_fake
def _(x_disp, W1_q, W1_scale, W2_q, W2_scale, lay, T, top_k, pad_multiple):
    return x_disp.new_empty(x_disp.shape)


def moe_layer_fp8_block(x: Tensor, topk_idx: Tensor, topk_probs: Tensor, W1_q: Tensor, W1_scale: Tensor, W2_q: Tensor,
                        W2_scale: Tensor, pad_multiple: int = 1, return_status: bool = False):
    """The layer for inference from weights with 128 x 128 block scales
    (quantize_fp8_block of W1 and W2, block_rows 128): multihot, dispatch,
    experts with both products in e4m3, combine.  Returns out, or with
    ``return_status`` (out, status) as moe_layer does."""
    T, K = topk_idx.shape
    E = W1_q.shape[0]
    rmap, probs, _, status = _ops.route_to_multihot(topk_idx, topk_probs, E)
    x_disp, *lay = _ops.dispatch(x, rmap, probs, status, K, pad_multiple)
    y = _ops.grouped_experts_fp8_block(x_disp, W1_q, W1_scale, W2_q, W2_scale, lay, T, K, pad_multiple)
    out = _ops.combine(y, lay, T, K, pad_multiple, E)
    return (out, lay[-1]) if return_status else out


def moe_block(x: Tensor, normed: Tensor, router: Tensor, top_k: int, W1: Tensor, W2: Tensor, norm_out_weight: Tensor,
              gate: Optional[Tensor] = None, next_weight: Optional[Tensor] = None, residual_scale: float = 1.0,
              pad_multiple: int = 1, eps: float = 1e-6, fp8: Optional[Tuple[Tensor, Tensor]] = None,
              return_status: bool = False):
    """A MoE block between two norms: from the residual stream x and its norm
    (``norm_in``, or the block before's ``next``), the router's logits
    ``normed @ router^T``, the layer, and ``norm_out``.  Returns (out, next), next
    being None without ``next_weight``, and with ``return_status`` the layer's
    status as a third.

    Differentiable in everything but the top-k choice.  With ``fp8`` = (W1_scale,
    W2_scale), W1 and W2 are e4m3 codes with block scales and the layer runs for
    inference."""
    logits = (normed.float() @ router.float().t()).contiguous()
    if fp8 is None:
        y, status = moe_layer_from_logits(normed, logits, top_k, W1, W2, pad_multiple, return_status=True)
    else:
        idx, p = _ops.router_topk(logits, top_k)
        y, status = moe_layer_fp8_block(normed, idx, p, W1, fp8[0], W2, fp8[1], pad_multiple, return_status=True)
    out, nxt, _, _ = _ops.norm_out(x, y, norm_out_weight, gate, next_weight, residual_scale, True, eps, 0.0)
    nxt = nxt if next_weight is not None else None
    return (out, nxt, status) if return_status else (out, nxt)


def moe_layer_from_logits(x: Tensor, router_logits: Tensor, top_k: int, W1: Tensor, W2: Tensor,
                          pad_multiple: int = 1, return_status: bool = False):
    """The router (softmax, top-k, renormalise) and the layer; gradients also
    reach the router logits."""
    topk_idx, topk_probs = torch.ops.moe_gb300.router_topk(router_logits, top_k)
    return moe_layer(x, topk_idx, topk_probs, W1, W2, pad_multiple, return_status)
