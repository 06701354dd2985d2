"""What stands around the MoE layer in a block: Python binding, argument checks only.

* moe_norm_in / moe_norm_out and their backwards: the RMS norms before and
  after a block, fused with its gate and residual scale;
* AdamWState / moe_adamw_step: the optimiser's step over many tensors at once,
  its averages in fp32 or in 8 bits;
* moe_quantize_fp8_block, moe_matmul_fp8_block and
  moe_grouped_experts_fp8_block: products of e4m3 codes with a scale for each
  block of 128.

As in ``moe.py`` the functions carry the names of the C entry points, all
arithmetic runs in the CUDA library, and PyTorch only allocates the buffers and
supplies the current stream.  Tensors are packed and on the GPU; anything
else is refused before a kernel is launched.  (Norm weights cut from a larger
buffer at any element are copied first, where the kernel wants whole vectors.)
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Union

import numpy as np
import torch

from . import _native as N
from . import moe as _m
from .moe import Layout, _check

_DTYPES = {torch.bfloat16: N.MOE_DTYPE_BF16, torch.float32: N.MOE_DTYPE_F32}
_GATES = {0: N.MOE_GATE_NONE, 1: N.MOE_GATE_TOKEN, 2: N.MOE_GATE_ELEMENT}


# The current stream's handle without a Python stream object around it: a
# call for one token is bound by what happens here on the host.
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _raw_stream(stream, device):
    """The handle of the stream to launch on.  A launch goes to the current
    device, so tensors and stream have to be there."""
    if device.index != _m._current_device():
        raise _m._wrong_device("the tensors are", device.index)
    if stream is None:
        return _current_raw_stream(device.index)
    if stream.device_index != device.index:
        raise _m._wrong_device("the stream is", stream.device_index)
    return stream.cuda_stream


def _used_on(stream, *made: Optional[torch.Tensor]):
    """Buffers made here for a call on a stream other than the current one:
    their memory is not given out again before that stream is done with it."""
    if stream is not None:
        for t in made:
            if t is not None and t.numel():
                t.record_stream(stream)


def _need(t: torch.Tensor, name: str, dtype, shape, device):
    """The address of a tensor that has to be as given (None for one without elements)."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr() or None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    raise ValueError(f"{name} must be contiguous")


def _vectors(w: Optional[torch.Tensor], stream):
    """A norm's weights at an address that rows of a multiple of 8 values allow: as they are, or a copy."""
    if w is None or w.data_ptr() % 16 == 0 or w.numel() % 8 or not w.is_contiguous() or not w.is_cuda:
        return w
    with torch.cuda.stream(stream):
        return w.detach().clone()


def _on_gpu(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device}): there is no CPU kernel")
    return t.device


def _either(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32 (got {t.dtype})")
    return code


def _rows(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T, H] (got {tuple(t.shape)})")
    return t.shape


def _norm(T, H, x, weight, gate, gate_sigmoid, residual_scale, eps, weight_offset, next_weight=None):
    if next_weight is not None and next_weight.dtype is not weight.dtype:
        raise TypeError("weight and next_weight must have the same type")
    if gate is not None and gate.shape != (T,) and gate.shape != (T, H):
        raise ValueError(f"gate must have shape {(T,)} or {(T, H)} (got {tuple(gate.shape)})")
    return N.MoeNorm(T, H, _either(x, "x"), _either(weight, "weight"),
                     N.MOE_DTYPE_F32 if gate is None else _either(gate, "gate"),
                     N.MOE_GATE_NONE if gate is None else _GATES[gate.dim()],
                     int(gate_sigmoid), residual_scale, eps, weight_offset)


@functools.lru_cache(maxsize=1024)
def _bytes(query: str, device: int, *sizes) -> int:
    """A workspace's size, which depends on its arguments and the device's SM
    count alone (``device``: the one that the call goes to)."""
    nbytes = ctypes.c_size_t(0)
    _check(getattr(N.lib, query)(*sizes, ctypes.byref(nbytes)), query)
    return nbytes.value


def _workspace(T, H, device):
    return torch.empty(_bytes("moe_norm_backward_workspace_bytes", device.index, T, H), dtype=torch.uint8, device=device)


def moe_norm_in(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, weight_offset: float = 0.0,
                save_rstd: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """The norm before a block: returns (norm [T, H] bf16, rstd fp32 [T] or
    None).  ``save_rstd`` keeps what moe_norm_in_backward needs."""
    T, H = _rows(x, "x")
    dev = _on_gpu(x, "x")
    weight = _vectors(weight, stream)
    n = _norm(T, H, x, weight, None, False, 1.0, eps, weight_offset)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev) if save_rstd else None
    _check(N.lib.moe_norm_in(n, _need(x, "x", x.dtype, (T, H), dev), _need(weight, "weight", weight.dtype, (H,), dev),
                             _need(out, "out", torch.bfloat16, (T, H), dev), rstd.data_ptr() or None if save_rstd else None,
                             _raw_stream(stream, dev)), "moe_norm_in")
    _used_on(stream, out, rstd)
    return out, rstd


def moe_norm_in_backward(grad_norm: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                         grad_res: Optional[torch.Tensor] = None, weight_offset: float = 0.0, stream=None):
    """Returns (grad_x [T, H] in x's type, grad_weight fp32 [H]).  ``grad_res``
    is the gradient that reaches x past the block; it is added to grad_x."""
    T, H = _rows(x, "x")
    dev = _on_gpu(x, "x")
    weight = _vectors(weight, stream)
    n = _norm(T, H, x, weight, None, False, 1.0, 0.0, weight_offset)
    grad_x = torch.empty(T, H, dtype=x.dtype, device=dev)
    grad_w = torch.empty(H, dtype=torch.float32, device=dev)
    ws = _workspace(T, H, dev)
    _check(N.lib.moe_norm_in_backward(
        n, _need(grad_norm, "grad_norm", torch.bfloat16, (T, H), dev), _need(x, "x", x.dtype, (T, H), dev),
        _need(weight, "weight", weight.dtype, (H,), dev), _need(rstd, "rstd", torch.float32, (T,), dev),
        None if grad_res is None else _need(grad_res, "grad_res", x.dtype, (T, H), dev),
        grad_x.data_ptr() or None, grad_w.data_ptr(), ws.data_ptr() or None, _raw_stream(stream, dev)),
        "moe_norm_in_backward")
    _used_on(stream, grad_x, grad_w, ws)
    return grad_x, grad_w


def moe_norm_out(x: torch.Tensor, y: torch.Tensor, weight: torch.Tensor, gate: Optional[torch.Tensor] = None,
                 residual_scale: float = 1.0, gate_sigmoid: bool = True, next_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, weight_offset: float = 0.0, save_rstd: bool = False, stream=None):
    """The norm after a block, its gate ([T] or [T, H]) and the residual:
    returns (out [T, H] in x's type, rstd or None, next [T, H] bf16 or None,
    next_rstd or None), next being the next block's norm of out."""
    T, H = _rows(x, "x")
    dev = _on_gpu(x, "x")
    weight, next_weight = _vectors(weight, stream), _vectors(next_weight, stream)
    n = _norm(T, H, x, weight, gate, gate_sigmoid, residual_scale, eps, weight_offset, next_weight)
    out = torch.empty(T, H, dtype=x.dtype, device=dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev) if save_rstd else None
    has_next = next_weight is not None
    nxt = torch.empty(T, H, dtype=torch.bfloat16, device=dev) if has_next else None
    next_rstd = torch.empty(T, dtype=torch.float32, device=dev) if save_rstd and has_next else None
    _check(N.lib.moe_norm_out(
        n, _need(x, "x", x.dtype, (T, H), dev), _need(y, "y", torch.bfloat16, (T, H), dev),
        _need(weight, "weight", weight.dtype, (H,), dev),
        None if gate is None else _need(gate, "gate", gate.dtype, gate.shape, dev), out.data_ptr() or None,
        rstd.data_ptr() or None if save_rstd else None,
        _need(next_weight, "next_weight", weight.dtype, (H,), dev) if has_next else None,
        nxt.data_ptr() or None if has_next else None,
        next_rstd.data_ptr() or None if next_rstd is not None else None, _raw_stream(stream, dev)), "moe_norm_out")
    _used_on(stream, out, rstd, nxt, next_rstd)
    return out, rstd, nxt, next_rstd


def moe_norm_out_backward(grad_out: Optional[torch.Tensor], y: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0, gate_sigmoid: bool = True,
                          grad_next: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          next_weight: Optional[torch.Tensor] = None, next_rstd: Optional[torch.Tensor] = None,
                          weight_offset: float = 0.0, stream=None):
    """Returns (grad_x, grad_y, grad_gate or None, grad_weight fp32 [H],
    grad_next_weight fp32 [H] or None).  With a next norm give grad_next, out,
    next_weight and next_rstd; grad_out may then be None."""
    T, H = _rows(y, "y")
    dev = _on_gpu(y, "y")
    has_next = next_weight is not None
    if any((t is not None) != has_next for t in (grad_next, out, next_rstd)):
        raise ValueError("give grad_next, out, next_weight and next_rstd, or none of them")
    if grad_out is None and not has_next:
        raise ValueError("grad_out may be None only with a next norm")
    stream_like = grad_out if grad_out is not None else out
    weight, next_weight = _vectors(weight, stream), _vectors(next_weight, stream)
    n = _norm(T, H, stream_like, weight, gate, gate_sigmoid, residual_scale, 0.0, weight_offset, next_weight)
    xt = stream_like.dtype
    grad_x = torch.empty(T, H, dtype=xt, device=dev)
    grad_y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    grad_gate = torch.empty_like(gate, memory_format=torch.contiguous_format) if gate is not None else None
    grad_w = torch.empty(H, dtype=torch.float32, device=dev)
    grad_w2 = torch.empty(H, dtype=torch.float32, device=dev) if has_next else None
    ws = _workspace(T, H, dev)
    _check(N.lib.moe_norm_out_backward(
        n, None if grad_out is None else _need(grad_out, "grad_out", xt, (T, H), dev),
        _need(grad_next, "grad_next", torch.bfloat16, (T, H), dev) if has_next else None,
        _need(out, "out", xt, (T, H), dev) if has_next else None, _need(y, "y", torch.bfloat16, (T, H), dev),
        _need(weight, "weight", weight.dtype, (H,), dev),
        None if gate is None else _need(gate, "gate", gate.dtype, gate.shape, dev),
        _need(rstd, "rstd", torch.float32, (T,), dev),
        _need(next_weight, "next_weight", weight.dtype, (H,), dev) if has_next else None,
        _need(next_rstd, "next_rstd", torch.float32, (T,), dev) if has_next else None,
        grad_x.data_ptr() or None, grad_y.data_ptr() or None, None if gate is None else grad_gate.data_ptr() or None,
        grad_w.data_ptr(), grad_w2.data_ptr() if has_next else None, ws.data_ptr() or None, _raw_stream(stream, dev)),
        "moe_norm_out_backward")
    _used_on(stream, grad_x, grad_y, grad_gate, grad_w, grad_w2, ws)
    return grad_x, grad_y, grad_gate, grad_w, grad_w2


# ------------------------------------------------------------------ AdamW
_TABLE = np.dtype([(n, {ctypes.c_void_p: np.uint64, ctypes.c_int64: np.int64, ctypes.c_int32: np.int32,
                        ctypes.c_double: np.float64}[c]) for n, c in N.MoeAdamwTensor._fields_])
assert _TABLE.itemsize == ctypes.sizeof(N.MoeAdamwTensor)


class AdamWState:
    """The parameters of an AdamW optimiser and its state, in caller-owned
    device buffers: for each parameter exp_avg and exp_avg_sq (fp32, or with
    state_bits=8 uint8 codes and one fp32 scale per 256 elements) and, with
    master=True, the fp32 value of which a bf16 parameter is the rounded copy.

    ``step`` counts the steps taken; ``seed`` draws the random rounding of 8-bit
    states.  The buffers may be given (to resume, or to place them): then
    they are used as they are, else they are made for a fresh start.  They stay
    the same for the state's life: load values into them with copy_."""

    def __init__(self, params: Sequence[torch.Tensor], state_bits: int = 32, master: Union[bool, Sequence, None] = None,
                 seed: int = 0, step: int = 0, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None,
                 exp_avg_sq_scale=None):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32 (got {state_bits})")
        if step < 0:
            raise ValueError(f"step must be >= 0 (got {step})")
        self.params = list(params)
        self.state_bits, self.seed, self.step = state_bits, seed & (2 ** 64 - 1), step
        eight = state_bits == 8
        for i, p in enumerate(self.params):
            _on_gpu(p, f"params[{i}]")
            _either(p, f"params[{i}]")
        if len({p.data_ptr() for p in self.params if p.numel()}) < sum(p.numel() > 0 for p in self.params):
            raise ValueError("params holds the same tensor twice")
        self.device = self.params[0].device if self.params else torch.device("cuda", torch.cuda.current_device())
        blocks = [-(-p.numel() // N.MOE_ADAMW_STATE_BLOCK) for p in self.params]

        def make(given, what, dtype, shapes):
            if given is None:
                return tuple(torch.zeros(s, dtype=dtype, device=self.device) for s in shapes)
            if len(given) != len(self.params):
                raise ValueError(f"{what} must hold one tensor per parameter")
            return tuple(given)

        shapes = [p.shape for p in self.params]
        avg = torch.uint8 if eight else torch.float32
        self._exp_avg = make(exp_avg, "exp_avg", avg, shapes)
        self._exp_avg_sq = make(exp_avg_sq, "exp_avg_sq", avg, shapes)
        self._exp_avg_scale = make(exp_avg_scale, "exp_avg_scale", torch.float32, blocks) if eight else None
        self._exp_avg_sq_scale = make(exp_avg_sq_scale, "exp_avg_sq_scale", torch.float32, blocks) if eight else None
        if isinstance(master, (list, tuple)):
            self._master = make(master, "master", torch.float32, shapes)
        else:
            self._master = tuple(p.detach().float() if p.dtype is torch.bfloat16 else None for p in self.params) \
                if master else None
        self._table = np.zeros(len(self.params), dtype=_TABLE)
        self._address = self._table.ctypes.data
        self._made_for = [(p.dtype, p.shape) for p in self.params]
        self._settings = None      # what the table's remaining columns were filled from
        for i, (p, row) in enumerate(zip(self.params, self._table)):
            row["n"], row["param_dtype"] = p.numel(), _either(p, f"params[{i}]")
            for name, dtype, shape in (("exp_avg", avg, p.shape), ("exp_avg_sq", avg, p.shape),
                                       ("exp_avg_scale", torch.float32, (blocks[i],)),
                                       ("exp_avg_sq_scale", torch.float32, (blocks[i],)),
                                       ("master", torch.float32, p.shape)):
                held = getattr(self, name)
                if held is not None and held[i] is not None:
                    row[name] = _need(held[i], f"{name}[{i}]", dtype, shape, self.device) or 0

    # (read-only: the table that the kernel gets was made from them)
    exp_avg = property(lambda self: self._exp_avg)
    exp_avg_sq = property(lambda self: self._exp_avg_sq)
    exp_avg_scale = property(lambda self: self._exp_avg_scale)
    exp_avg_sq_scale = property(lambda self: self._exp_avg_sq_scale)
    master = property(lambda self: self._master)


def moe_adamw_step(state: AdamWState, grads: Sequence[Optional[torch.Tensor]], lr: float, beta1: float = 0.9,
                   beta2: float = 0.999, eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.0,
                   grad_scale: Optional[torch.Tensor] = None, skip: Optional[torch.Tensor] = None,
                   step: Optional[torch.Tensor] = None, stream=None) -> None:
    """One step, in place, over all of ``state``'s parameters in one launch (one
    per 96 tensors).  A gradient is bf16 or fp32 in its parameter's shape; a
    parameter whose gradient is None is left as it is.  ``weight_decay`` is one
    number or one per parameter.

    On the device: ``grad_scale`` fp32 [1] multiplies every gradient (an
    unscaling or a clip that the host need not know), ``skip`` int32 [1] turns
    the step into a no-op when it is not zero, and ``step`` int64 [1] replaces
    state.step + 1, for a captured call whose step number changes between
    replays.  Without ``step``, state.step is counted up here -- also when
    ``skip`` stops the update, which only the device knows."""
    params, table, dev = state.params, state._table, state.device
    if len(grads) != len(params):
        raise ValueError(f"{len(grads)} gradients for {len(params)} parameters")
    if params:
        places, addresses, dtypes = [], [], []
        for p, g, (dtype, shape) in zip(params, grads, state._made_for):
            if p.dtype is not dtype or p.shape != shape or p.device != dev or not p.is_contiguous():
                raise ValueError(f"params[{len(places)}] is no longer what the state was made for")
            places.append(p.data_ptr())
            if g is None:
                addresses.append(0)
                dtypes.append(None)
                continue
            if g.shape != shape or g.device != dev or not g.is_contiguous():
                _need(g, f"grads[{len(addresses)}]", g.dtype, shape, dev)   # says which
            addresses.append(g.data_ptr())
            dtypes.append(g.dtype)
        table["param"], table["grad"] = places, addresses
        # only the addresses change in most steps
        if not isinstance(weight_decay, (int, float)):
            weight_decay = [float(d) for d in weight_decay]
            if len(weight_decay) != len(params):
                raise ValueError(f"{len(weight_decay)} weight decays for {len(params)} parameters")
        settings = (dtypes, weight_decay)
        if settings != state._settings:
            state._settings = None
            table["grad_dtype"] = [0 if g is None else _either(g, f"grads[{i}]") for i, g in enumerate(grads)]
            table["n"] = [0 if g is None else g.numel() for g in grads]
            table["weight_decay"] = weight_decay
            state._settings = settings
    scalar = [None if t is None else _need(t, name, dtype, (1,), dev)
              for t, name, dtype in ((grad_scale, "grad_scale", torch.float32), (skip, "skip", torch.int32),
                                     (step, "step", torch.int64))]
    h = N.MoeAdamw(lr, beta1, beta2, eps, state.step + 1, state.seed, state.state_bits, *scalar)
    _check(N.lib.moe_adamw_step(h, state._address, len(params), _raw_stream(stream, dev)), "moe_adamw_step")
    if step is None:
        state.step += 1
    if params:
        torch.autograd.graph.increment_version(params)


# ------------------------------------------------------------------ e4m3 with a scale per block of 128
def _blocks(n: int) -> int:
    return -(-n // 128)


def moe_quantize_fp8_block(src: torch.Tensor, block_rows: int = 1, out=None, stream=None):
    """e4m3 codes of a bf16 tensor [..., rows, cols] (uint8, same shape) and fp32
    scales [..., ceil(rows / block_rows), ceil(cols / 128)]: block_rows=1 for
    activations, 128 for weights.  cols is a multiple of 16."""
    dev = _on_gpu(src, "src")
    if src.dim() < 2:
        raise ValueError(f"src must be [..., rows, cols] (got {tuple(src.shape)})")
    rows, cols = src.shape[-2:]
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128 (got {block_rows})")
    lead = src.shape[:-2]
    batch = lead.numel() if lead else 1
    shape = (*lead, -(-rows // block_rows), _blocks(cols))
    if out is None:
        out = (torch.empty(src.shape, dtype=torch.uint8, device=dev), torch.empty(shape, dtype=torch.float32, device=dev))
    codes, scales = out
    _check(N.lib.moe_quantize_fp8_block(_need(src, "src", torch.bfloat16, src.shape, dev), batch, rows, cols, block_rows,
                                        _need(codes, "codes", torch.uint8, src.shape, dev),
                                        _need(scales, "scales", torch.float32, shape, dev), _raw_stream(stream, dev)),
           "moe_quantize_fp8_block")
    _used_on(stream, codes, scales)
    return codes, scales


def moe_matmul_fp8_block(a_q: torch.Tensor, a_scale: torch.Tensor, b_q: torch.Tensor, b_scale: torch.Tensor,
                         out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """a b^T of codes [M, K] and [N, K] with their scales (block_rows 1 and 128):
    [M, N] bf16."""
    dev = _on_gpu(a_q, "a_q")
    M, K = _rows(a_q, "a_q")
    n = _rows(b_q, "b_q")[0]
    if out is None:
        out = torch.empty(M, n, dtype=torch.bfloat16, device=dev)
    kb = _blocks(K)
    _check(N.lib.moe_matmul_fp8_block(_need(a_q, "a_q", torch.uint8, (M, K), dev),
                                      _need(a_scale, "a_scale", torch.float32, (M, kb), dev), M,
                                      _need(b_q, "b_q", torch.uint8, (n, K), dev),
                                      _need(b_scale, "b_scale", torch.float32, (_blocks(n), kb), dev), n, K,
                                      _need(out, "out", torch.bfloat16, (M, n), dev),
                                      None if status is None else _need(status, "status", torch.int32, (1,), dev),
                                      _raw_stream(stream, dev)), "moe_matmul_fp8_block")
    _used_on(stream, out)
    return out


def moe_grouped_experts_fp8_block(x_disp: torch.Tensor, layout: Layout, W1_q: torch.Tensor, W1_scale: torch.Tensor,
                                  W2_q: torch.Tensor, W2_scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                                  stream=None):
    """The grouped SwiGLU experts from e4m3 weights with 128 x 128 block scales:
    y [C, H] bf16 with the routing weights applied, for moe_combine."""
    dev = _on_gpu(x_disp, "x_disp")
    C, H = layout.capacity, _rows(x_disp, "x_disp")[1]
    if W1_q.dim() != 3 or W1_q.shape[1] % 2:
        raise ValueError(f"W1_q must be [E, 2I, H] (got {tuple(W1_q.shape)})")
    E, I = layout.E, W1_q.shape[1] // 2
    if out is None:
        out = torch.empty(C, H, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(_bytes("moe_experts_fp8_block_workspace_bytes", dev.index, C, layout.T, E, H, I), dtype=torch.uint8,
                     device=dev)
    _check(N.lib.moe_grouped_experts_fp8_block(
        _need(x_disp, "x_disp", torch.bfloat16, (C, H), dev), layout.ref, H, I,
        _need(W1_q, "W1_q", torch.uint8, (E, 2 * I, H), dev),
        _need(W1_scale, "W1_scale", torch.float32, (E, _blocks(2 * I), _blocks(H)), dev),
        _need(W2_q, "W2_q", torch.uint8, (E, H, I), dev),
        _need(W2_scale, "W2_scale", torch.float32, (E, _blocks(H), _blocks(I)), dev),
        _need(out, "out", torch.bfloat16, (C, H), dev), ws.data_ptr() or None, _raw_stream(stream, dev)),
        "moe_grouped_experts_fp8_block")
    _used_on(stream, out, ws)
    return out
