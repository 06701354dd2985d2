"""The operators around the layer without a GPU: fake shapes, tracing of a whole
block, loud failure on CPU tensors, and the refusals of the C ABI."""
import ctypes

import pytest
import torch
from torch.fx.experimental.proxy_tensor import make_fx

import combine_topk_multihot_gb300 as moe
from combine_topk_multihot_gb300 import _native as N, ops

T, H, E, K, I = 64, 256, 8, 2, 128


def _inputs(device, grad=True):
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    t = dict(x=mk(T, H), normed=mk(T, H), router=mk(E, H), W1=mk(E, 2 * I, H), W2=mk(E, H, I),
             w=mk(H, dt=torch.float32), gate=mk(T, dt=torch.float32), w2=mk(H, dt=torch.float32))
    return {k: v.requires_grad_(grad) for k, v in t.items()}


def _block(t, **kw):
    return ops.moe_block(t["x"], t["normed"], t["router"], K, t["W1"], t["W2"], t["w"], gate=t["gate"],
                         next_weight=t["w2"], **kw)


def test_fake_shapes_and_gradients():
    t = _inputs("meta")
    out, nxt = _block(t)
    assert out.shape == nxt.shape == (T, H) and out.dtype == nxt.dtype == torch.bfloat16
    (out.float().sum() + nxt.float().sum()).backward()
    assert all(v.grad is not None and v.grad.shape == v.shape and v.grad.dtype == v.dtype for v in t.values())


def test_trace_holds_the_operators():
    t = _inputs("cpu", grad=False)
    gm = make_fx(lambda *a: _block(dict(zip(t, a))), tracing_mode="symbolic")(*t.values())
    used = {str(n.target).split(".")[1] for n in gm.graph.nodes
            if n.op == "call_function" and str(n.target).startswith("moe_gb300.")}
    assert used == {"router_topk", "route_to_multihot", "dispatch", "grouped_experts", "combine", "norm_out"}


def test_fp8_block_trace():
    t = _inputs("meta", grad=False)
    u8 = lambda s: torch.zeros(s, dtype=torch.uint8, device="meta")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="meta")  # noqa: E731
    t["W1"], t["W2"] = u8(t["W1"].shape), u8(t["W2"].shape)
    out, nxt = _block(t, fp8=(f32(E, 2, 2), f32(E, 2, 1)))
    assert out.shape == nxt.shape == (T, H)
    q, s = torch.ops.moe_gb300.quantize_fp8_block(torch.zeros(3, 200, 144, dtype=torch.bfloat16, device="meta"), 128)
    assert q.shape == (3, 200, 144) and s.shape == (3, 2, 2)


def test_cpu_tensors_fail_loudly():
    t = _inputs("cpu", grad=False)
    with pytest.raises(NotImplementedError, match="CPU"):
        torch.ops.moe_gb300.norm_in(t["x"], t["w"], 1e-6, 0.0)
    with pytest.raises(ValueError, match="GPU"):
        moe.AdamWState([t["w"]])


P = ctypes.c_void_p
OK, ODD = P(256), P(256 + 4)     # never dereferenced: validation fails first


def _norm(**kw):
    d = dict(T=4, H=64, x_dtype=0, weight_dtype=1, gate_dtype=1, gate_kind=0, gate_sigmoid=1, residual_scale=1.0, eps=1e-6,
             weight_offset=0.0)
    d.update(kw)
    return N.MoeNorm(*(d[f] for f, _ in N.MoeNorm._fields_))


def test_norm_validation():
    call = lambda n, *p: N.lib.moe_norm_in(n, *p, None)  # noqa: E731
    assert call(None, OK, OK, OK, None) == N.MOE_ERR_INVALID_ARG
    assert call(_norm(), None, OK, OK, None) == N.MOE_ERR_INVALID_ARG
    assert call(_norm(), OK, ODD, OK, None) == N.MOE_ERR_INVALID_ARG
    for bad in (dict(T=-1), dict(x_dtype=2), dict(gate_kind=3), dict(eps=-1.0), dict(eps=float("nan")),
                dict(residual_scale=float("inf"))):
        assert call(_norm(**bad), OK, OK, OK, None) == N.MOE_ERR_INVALID_ARG, bad
    for H in (0, 16385):
        assert call(_norm(H=H), OK, OK, OK, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
    # norm_out: the gate and the next norm come whole or not at all
    out = lambda n, gate, w2, nx, r2: N.lib.moe_norm_out(n, OK, OK, OK, gate, OK, None, w2, nx, r2, None)  # noqa: E731
    assert out(_norm(), OK, None, None, None) == N.MOE_ERR_INVALID_ARG
    assert out(_norm(gate_kind=1), None, None, None, None) == N.MOE_ERR_INVALID_ARG
    assert out(_norm(), None, OK, None, None) == N.MOE_ERR_INVALID_ARG
    assert out(_norm(), None, None, None, OK) == N.MOE_ERR_INVALID_ARG
    back = lambda n, go, gn, w2: N.lib.moe_norm_out_backward(  # noqa: E731
        n, go, gn, OK, OK, OK, None, OK, OK, OK, OK, OK, None, OK, w2, OK, None)
    assert back(_norm(), OK, None, OK) == N.MOE_ERR_INVALID_ARG          # grad_next missing
    assert back(_norm(), OK, OK, None) == N.MOE_ERR_INVALID_ARG          # grad_next without its weight's gradient
    n = ctypes.c_size_t(0)
    assert N.lib.moe_norm_backward_workspace_bytes(-1, 64, ctypes.byref(n)) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_norm_backward_workspace_bytes(0, 64, ctypes.byref(n)) == 0 and n.value == 0


def test_adamw_validation():
    def call(h=None, t=None, count=1):
        a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=0, state_bits=32, grad_scale=None, skip=None,
                 step_dev=None)
        a.update(h or {})
        b = dict(param=256, grad=256, master=None, exp_avg=256, exp_avg_sq=256, exp_avg_scale=None, exp_avg_sq_scale=None,
                 n=8, param_dtype=1, grad_dtype=1, weight_decay=0.0)
        b.update(t or {})
        return N.lib.moe_adamw_step(N.MoeAdamw(*a.values()), ctypes.byref(N.MoeAdamwTensor(*b.values())), count, None)

    for h in (dict(state_bits=16), dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(lr=-1.0), dict(lr=float("inf")),
              dict(eps=float("nan")), dict(skip=258), dict(step_dev=260)):
        assert call(h) == N.MOE_ERR_INVALID_ARG, h
    for t in (dict(n=-1), dict(param=None), dict(grad=None), dict(param_dtype=2), dict(master=256), dict(grad=258),
              dict(weight_decay=-1.0)):
        assert call(None, t) == N.MOE_ERR_INVALID_ARG, t
    assert call(dict(state_bits=8)) == N.MOE_ERR_INVALID_ARG             # no scales
    assert call(None, dict(n=1 << 40)) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(None, None, -1) == N.MOE_ERR_INVALID_ARG


def test_fp8_block_validation():
    q = lambda *a: N.lib.moe_quantize_fp8_block(OK, *a, OK, OK, None)  # noqa: E731
    assert q(1, 4, 24, 1) == N.MOE_ERR_UNSUPPORTED_SHAPE and q(1, 4, 0, 1) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(1, 4, 32, 2) == N.MOE_ERR_INVALID_ARG and q(-1, 4, 32, 1) == N.MOE_ERR_INVALID_ARG
    assert q(1 << 20, 1 << 20, 256, 1) == N.MOE_ERR_UNSUPPORTED_SHAPE
    mm = lambda M, n, k, a=OK: N.lib.moe_matmul_fp8_block(a, OK, M, OK, OK, n, k, OK, None, None)  # noqa: E731
    assert mm(-1, 8, 128) == N.MOE_ERR_INVALID_ARG and mm(4, 0, 128) == N.MOE_ERR_INVALID_ARG
    assert mm(4, 8, 120) == N.MOE_ERR_UNSUPPORTED_SHAPE and mm(4, 8, 128, None) == N.MOE_ERR_INVALID_ARG
    assert mm(4, 8, 128, ODD) == N.MOE_ERR_INVALID_ARG
    L = N.MoeLayout(4, 8, 2, 1, 8)
    assert N.lib.moe_grouped_experts_fp8_block(OK, ctypes.byref(L), 256, 128, OK, OK, OK, OK, OK, OK, None) == \
        N.MOE_ERR_INVALID_ARG                                            # the layout's pointers are NULL


def test_status_is_returned_on_request():
    t = _inputs("meta", grad=False)
    assert len(_block(t)) == 2
    out, nxt, status = _block(t, return_status=True)
    assert out.shape == nxt.shape == (T, H) and status.shape == (1,) and status.dtype == torch.int32
    u8 = lambda s: torch.zeros(s, dtype=torch.uint8, device="meta")  # noqa: E731
    q1, q2, s1, s2 = u8(t["W1"].shape), u8(t["W2"].shape), torch.zeros(E, 2, 2, device="meta"), torch.zeros(E, 2, 1, device="meta")
    idx, p = torch.zeros(T, K, dtype=torch.int64, device="meta"), torch.zeros(T, K, device="meta")
    assert torch.is_tensor(ops.moe_layer_fp8_block(t["x"], idx, p, q1, s1, q2, s2))
    out, status = ops.moe_layer_fp8_block(t["x"], idx, p, q1, s1, q2, s2, return_status=True)
    assert out.shape == (T, H) and status.shape == (1,) and status.dtype == torch.int32


def test_alignment_by_what_is_read():
    """What a kernel reads value by value needs no more than its type's alignment;
    validation alone: without a GPU what passes it ends with a device error."""
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real: nothing may be launched")
    refused, two = N.MOE_ERR_INVALID_ARG, P(256 + 2)
    x8, x7 = _norm(H=64), _norm(H=63)
    norm_in = lambda n, x, w, o, r: N.lib.moe_norm_in(n, x, w, o, r, None)  # noqa: E731
    assert norm_in(x8, OK, OK, OK, ODD) != refused and norm_in(x8, OK, OK, OK, two) == refused
    for at in range(3):
        ptrs = [OK, OK, OK]
        ptrs[at] = ODD
        assert norm_in(x8, *ptrs, None) == refused and norm_in(x7, *ptrs, None) != refused
    assert norm_in(x7, OK, two, OK, None) == refused            # fp32 weights
    out = lambda n, gate: N.lib.moe_norm_out(n, OK, OK, OK, gate, OK, None, None, None, None, None)  # noqa: E731
    assert out(_norm(gate_kind=1), ODD) != refused and out(_norm(gate_kind=1), two) == refused
    assert out(_norm(gate_kind=1, gate_dtype=0), two) != refused
    assert out(_norm(gate_kind=2), ODD) == refused and out(_norm(gate_kind=2, H=63), ODD) != refused
    mm = lambda n, sa, sb, o: N.lib.moe_matmul_fp8_block(OK, sa, 4, OK, sb, n, 128, o, None, None)  # noqa: E731
    assert mm(8, ODD, ODD, OK) != refused and mm(8, two, OK, OK) == refused
    assert mm(8, OK, OK, two) == refused and mm(9, OK, OK, two) != refused
    assert N.lib.moe_quantize_fp8_block(OK, 1, 4, 128, 1, OK, ODD, None) != refused


def test_adamw_divisor_stays_in_range():
    """An eps for which the update's fast division would leave its range is refused."""
    def call(eps):
        h = N.MoeAdamw(1e-3, 0.9, 0.99, eps, 1, 0, 32, None, None, None)
        return N.lib.moe_adamw_step(h, None, 0, None)

    for eps in (1e30, 1e38, float("inf"), float("nan"), -1e-8):
        assert call(eps) == N.MOE_ERR_INVALID_ARG
        assert "eps" in N.last_error()
    assert call(9e29) != N.MOE_ERR_INVALID_ARG      # (without a GPU: a device error)
