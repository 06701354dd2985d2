"""The norms before and after a block against plain fp64 formulas.

Tolerances.  u = 2^-24 is the fp32 unit roundoff, 2^-9 half a bf16 ulp
relative to its value.  A row sum of H products in fp32 by threads of at most
64 sequential terms, then a tree, is off by at most (64 + 20) u times the sum
of the terms' magnitudes; an element takes about 20 more fp32 operations.  So
fp32 outputs are held to 256 u of the sum of the magnitudes of the terms that
make them up (their formula with every term replaced by its absolute value),
and bf16 outputs to that plus 2^-8 (1 + 2^-8) of their own magnitude: half an
ulp is at most 2^-8 relative to the value.  The weights' gradients add T terms
in fp32, at most ceil(T / rows a CTA) + 40 of them one after the other: 64 u
more suffice for the T here.  Where the next norm reads a stream rounded to
bf16, the oracle reads the GPU's own rounded stream.
"""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_multihot_gb300 as m
    return m


def _randn(g, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(DEV)


def _close(got, ref, magnitude, what):
    assert got.shape == ref.shape, what
    got64 = got.double()
    tol = 320 * U * magnitude + 1e-30
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -8) * ref.abs() + 2.0 ** -133
    bad = ~((got64 - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {((got64 - ref).abs() / tol).max():.3g} tol"


def _rms64(v, eps):
    return (v.square().mean(-1, keepdim=True) + eps).rsqrt()


# ragged and odd widths, one value, one vector, every vectors-per-thread form
SIZES = [(1, 1), (1, 2048), (3, 7), (5, 8), (2, 33), (130, 256), (33, 2048), (7, 2049), (700, 512), (9, 4096),
         (400, 4096), (5, 4104), (320, 8192), (4, 8199), (3, 16384), (310, 10000),
         # rows for every SM: through shared memory, in groups of 32 to 512 threads
         (1300, 264), (1300, 1024), (2000, 2048), (1300, 4096), (640, 5000), (650, 8192), (640, 16384),
         # and rows that do not start on 16 bytes
         (1300, 130), (1300, 2049), (640, 8199)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,wt", [(BF16, F32), (F32, BF16)])
def test_norm_in(moe, T, H, xt, wt):
    g = torch.Generator().manual_seed(T * 7 + H)
    x, w = _randn(g, T, H, dtype=xt, std=3.0), _randn(g, H, dtype=wt)
    n, rstd = moe.moe_norm_in(x, w, eps=1e-5, weight_offset=1.0, save_rstd=True)
    r = _rms64(x.double(), 1e-5)
    ref = x.double() * r * (1.0 + w.double())
    _close(n, ref, (x.double() * r).abs() * (1.0 + w.double().abs()), "norm")
    _close(rstd, r[:, 0], r[:, 0], "rstd")
    dn, dres = _randn(g, T, H, dtype=BF16), _randn(g, T, H, dtype=xt)
    for res in (dres, None):
        gx, gw = moe.moe_norm_in_backward(dn, x, w, rstd, grad_res=res, weight_offset=1.0)
        dx, dw, mx, mw = _norm_vjp(x, rstd, w.double() + 1.0, w.double().abs() + 1.0, dn)
        base = res.double() if res is not None else 0.0
        _close(gx, base + dx, mx + (res.double().abs() if res is not None else 0.0), "grad_x")
        _close(gw, dw, mw, "grad_weight")


def _norm_vjp(x, rstd, w, w_abs, dn):
    """(dx, dw) of x r w for the gradient dn, and the sums of their terms' magnitudes."""
    x, r, dn = x.double(), rstd.double()[:, None], dn.double()
    e, ea = w * dn, w_abs * dn.abs()
    dx = r * e - x * r ** 3 * (e * x).mean(-1, keepdim=True)
    mx = r * ea + x.abs() * r ** 3 * (ea * x.abs()).mean(-1, keepdim=True)
    return dx, (dn * x * r).sum(0), mx, (dn * x * r).abs().sum(0)


CASES = [(T, H, xt, gate, nxt) for (T, H), (xt, gate, nxt) in zip(
    itertools.cycle(SIZES), itertools.product((BF16, F32), ("none", "token", "element"), (False, True)))]
CASES += [(T, H, BF16, "token", True) for T, H in SIZES] + [(T, H, F32, "element", True) for T, H in SIZES]


@pytest.mark.parametrize("T,H,xt,gate_kind,has_next", CASES)
@pytest.mark.parametrize("sigmoid,gt", [(True, BF16), (False, F32)])
def test_norm_out(moe, T, H, xt, gate_kind, has_next, sigmoid, gt):
    g = torch.Generator().manual_seed(T * 3 + H)
    x, y = _randn(g, T, H, dtype=xt, std=2.0), _randn(g, T, H, dtype=BF16, std=0.3)
    w, w2 = _randn(g, H, mean=1.0, std=0.2), _randn(g, H, mean=1.0, std=0.2)
    gate = {"none": None, "token": _randn(g, T, dtype=gt), "element": _randn(g, T, H, dtype=gt, std=3.0)}[gate_kind]
    kw = dict(gate=gate, residual_scale=0.7, gate_sigmoid=sigmoid)
    out, rstd, nxt, rstd2 = moe.moe_norm_out(x, y, w, next_weight=w2 if has_next else None, eps=1e-6, save_rstd=True, **kw)
    y64, w64, r = y.double(), w.double(), _rms64(y.double(), 1e-6)
    s = torch.ones(T, 1, dtype=torch.float64, device=DEV)
    if gate is not None:
        s = (torch.sigmoid(gate.double()) if sigmoid else gate.double()).view(T, -1)
    hat = y64 * r * w64
    _close(out, 0.7 * x.double() + s * hat, (0.7 * x.double()).abs() + (s * hat).abs(), "out")
    _close(rstd, r[:, 0], r[:, 0], "rstd")
    if has_next:
        o = out.double()
        r2 = _rms64(o, 1e-6)
        _close(nxt, o * r2 * w2.double(), (o * r2 * w2.double()).abs(), "next")
        _close(rstd2, r2[:, 0], r2[:, 0], "next_rstd")
        sep, sep_r = moe.moe_norm_in(out, w2, eps=1e-6, save_rstd=True)   # the fused norm is the separate call's
        _close(nxt, sep.double(), sep.double().abs(), "next against moe_norm_in")

    dout, dnext = _randn(g, T, H, dtype=xt), _randn(g, T, H, dtype=BF16)
    back = dict(grad_next=dnext, out=out, next_weight=w2, next_rstd=rstd2) if has_next else {}
    for go in ((dout, None) if has_next else (dout,)):
        gx, gy, gg, gw, gw2 = moe.moe_norm_out_backward(go, y, w, rstd, **kw, **back)
        d = go.double() if go is not None else torch.zeros(T, H, dtype=torch.float64, device=DEV)
        md = d.abs()
        if has_next:
            dd, dw2, mdd, mw2 = _norm_vjp(out, rstd2, w2.double(), w2.double().abs(), dnext)
            d, md = d + dd, md + mdd
            _close(gw2, dw2, mw2, "grad_next_weight")
        _close(gx, 0.7 * d, 0.7 * md, "grad_x")
        r64 = rstd.double()[:, None]
        hat = y64 * r64
        slope = s * (1 - s) if sigmoid else torch.ones_like(s)
        if gate_kind == "element":
            _close(gg, slope * d * hat * w64, (slope * md * hat * w64).abs(), "grad_gate")
        elif gate_kind == "token":
            _close(gg, slope[:, 0] * (d * hat * w64).sum(1), slope[:, 0].abs() * (md * (hat * w64).abs()).sum(1), "grad_gate")
        else:
            assert gg is None
        e, me = w64 * s * d, (w64 * s).abs() * md
        _close(gy, r64 * e - y64 * r64 ** 3 * (e * y64).mean(1, keepdim=True),
               r64 * me + y64.abs() * r64 ** 3 * (me * y64.abs()).mean(1, keepdim=True), "grad_y")
        _close(gw, (s * d * hat).sum(0), (s.abs() * md * hat.abs()).sum(0), "grad_weight")


def test_backward_against_differences(moe):
    """The whole chain norm_out -> next norm as a function of each input, by
    central differences of the fp64 formulas along random directions."""
    g = torch.Generator().manual_seed(5)
    T, H, h = 6, 96, 1e-5
    x, y = _randn(g, T, H), _randn(g, T, H, dtype=BF16)
    w, w2, gate = _randn(g, H), _randn(g, H), _randn(g, T)
    dout, dnext = _randn(g, T, H), _randn(g, T, H, dtype=BF16)
    out, rstd, nxt, rstd2 = moe.moe_norm_out(x, y, w, gate=gate, residual_scale=0.7, next_weight=w2, save_rstd=True)
    gx, gy, gg, gw, gw2 = moe.moe_norm_out_backward(dout, y, w, rstd, gate=gate, residual_scale=0.7, grad_next=dnext,
                                                    out=out, next_weight=w2, next_rstd=rstd2)

    def loss(x, y, w, gate, w2):
        o = 0.7 * x + torch.sigmoid(gate)[:, None] * (y * _rms64(y, 1e-6) * w)
        return (o * dout.double()).sum() + (o * _rms64(o, 1e-6) * w2 * dnext.double()).sum()

    args = [t.double() for t in (x, y, w, gate, w2)]
    for k, grad in enumerate((gx, gy, gw, gg, gw2)):
        dirn = torch.randn(args[k].shape, generator=g, dtype=torch.float64).to(DEV)
        plus, minus = list(args), list(args)
        plus[k], minus[k] = args[k] + h * dirn, args[k] - h * dirn
        num = (loss(*plus) - loss(*minus)) / (2 * h)
        ana = (grad.double() * dirn).sum()
        # the differences: h^2 and 1e-16 / h; the gradients: fp32, or 2^-9 an element of grad_y's random sum
        scale = (grad.double() * dirn).norm()
        assert (num - ana).abs() <= scale * (0.02 if k == 1 else 1e-4) + 1e-6, (k, num, ana)


def test_no_rows(moe):
    x, w = torch.empty(0, 64, dtype=BF16, device=DEV), torch.ones(64, device=DEV)
    n, rstd = moe.moe_norm_in(x, w, save_rstd=True)
    assert n.shape == (0, 64) and rstd.shape == (0,)
    gx, gw = moe.moe_norm_in_backward(x, x, w, rstd)
    assert gx.shape == (0, 64) and torch.equal(gw, torch.zeros(64, device=DEV))
    out, r, nx, r2 = moe.moe_norm_out(x, x, w, next_weight=w, save_rstd=True)
    got = moe.moe_norm_out_backward(out, x, w, r, grad_next=nx, out=out, next_weight=w, next_rstd=r2)
    assert torch.equal(got[3], torch.zeros(64, device=DEV)) and torch.equal(got[4], torch.zeros(64, device=DEV))


def test_special_values(moe):
    """A row of zeros, a row with an infinity and one with NaN do what the
    formula says and leave the other rows alone."""
    g = torch.Generator().manual_seed(1)
    x, w = _randn(g, 5, 256, dtype=BF16), torch.ones(256, device=DEV)
    clean, _ = moe.moe_norm_in(x, w)
    x[1] = 0
    x[2, 3] = float("inf")
    x[3, 250] = float("nan")
    n, rstd = moe.moe_norm_in(x, w, eps=1e-6, save_rstd=True)
    assert torch.equal(n[0], clean[0]) and torch.equal(n[4], clean[4])
    assert (n[1] == 0).all() and abs(float(rstd[1]) - 1e3) < 1e-3
    assert float(rstd[2]) == 0 and n[2, 3].isnan() and (n[2, :3] == 0).all()
    assert n[3].isnan().all()


def test_repeats_and_other_stream(moe):
    """Same bits on every run, and on a stream other than the current one."""
    g = torch.Generator().manual_seed(2)
    T, H = 3001, 1536
    y, d, w = _randn(g, T, H, dtype=BF16), _randn(g, T, H, dtype=BF16), _randn(g, H)
    rstd = torch.rand(T, generator=g).to(DEV)
    first = moe.moe_norm_out_backward(d, y, w, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        again = moe.moe_norm_out_backward(d, y, w, rstd, stream=side)
        side.synchronize()
        for a, b in zip(first, again):
            assert (a is None and b is None) or torch.equal(a, b)


def test_scratch_of_another_stream_is_not_given_out(moe):
    """A call on a busy side stream, then allocations on the current one that
    would get its scratch: they must not disturb it."""
    g = torch.Generator().manual_seed(7)
    T, H = 2000, 2048
    y, d, w = _randn(g, T, H, dtype=BF16), _randn(g, T, H, dtype=BF16), _randn(g, H)
    rstd = torch.rand(T, generator=g).to(DEV)
    first = moe.moe_norm_out_backward(d, y, w, rstd)
    torch.cuda.synchronize()
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(8):
                a = torch.tanh(a @ a)          # keeps the side stream busy for a while
        again = moe.moe_norm_out_backward(d, y, w, rstd, stream=side)
        for n in (1 << 20, 1 << 21, 1 << 22, 1 << 23):
            torch.empty(n, device=DEV).fill_(float("nan"))
        side.synchronize()
        assert torch.equal(first[3], again[3]) and torch.equal(first[1], again[1])


def test_captured(moe):
    """A captured call reads its inputs anew at each replay."""
    g = torch.Generator().manual_seed(3)
    x, y, w = _randn(g, 200, 512, dtype=BF16), _randn(g, 200, 512, dtype=BF16), _randn(g, 512)
    moe.moe_norm_out(x, y, w, next_weight=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, nxt, _ = moe.moe_norm_out(x, y, w, next_weight=w)
    y.copy_(_randn(g, 200, 512, dtype=BF16))
    graph.replay()
    torch.cuda.synchronize()
    ref = moe.moe_norm_out(x, y, w, next_weight=w)
    assert torch.equal(out, ref[0]) and torch.equal(nxt, ref[2])


def test_refusals(moe):
    x, w = torch.zeros(4, 64, dtype=BF16, device=DEV), torch.ones(64, device=DEV)
    r = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_norm_in(x.cpu(), w)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        moe.moe_norm_in(x.half(), w)
    with pytest.raises(ValueError, match="weight must have shape"):
        moe.moe_norm_in(x, w[:32])
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_norm_in(torch.zeros(64, 4, dtype=BF16, device=DEV).t(), w)
    with pytest.raises(ValueError, match="on cuda"):
        moe.moe_norm_in(x, w.cpu())
    with pytest.raises(TypeError, match="y must be"):
        moe.moe_norm_out(x, x.float(), w)
    with pytest.raises(ValueError, match="gate must have shape"):
        moe.moe_norm_out(x, x, w, gate=torch.zeros(5, device=DEV))
    with pytest.raises(TypeError, match="same type"):
        moe.moe_norm_out(x, x, w, next_weight=w.bfloat16())
    with pytest.raises(ValueError, match="or none of them"):
        moe.moe_norm_out_backward(x, x, w, r, grad_next=x)
    with pytest.raises(ValueError, match="only with a next norm"):
        moe.moe_norm_out_backward(None, x, w, r)
    with pytest.raises(moe.MoEError, match="eps"):
        moe.moe_norm_in(x, w, eps=-1.0)
    with pytest.raises(moe.MoEError, match="16-byte"):
        moe.moe_norm_in(torch.zeros(4 * 64 + 1, dtype=BF16, device=DEV)[1:].view(4, 64), w)
    with pytest.raises(moe.MoEError, match="16384"):
        moe.moe_norm_in(torch.zeros(1, 16385, dtype=BF16, device=DEV), torch.ones(16385, device=DEV))


# rows enough for a third CTA an SM in the backward of the forms with few row tensors
@pytest.mark.parametrize("T,H", [(5600, 2560), (11200, 2048)])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_many_rows(moe, T, H, xt):
    test_norm_in(moe, T, H, xt, F32)
    for gate_kind, gt in (("none", F32), ("token", BF16)):
        test_norm_out(moe, T, H, xt, gate_kind, False, True, gt)


@pytest.mark.parametrize("H", [264, 384, 512])
def test_one_warp_a_row(moe, H):
    """Rows that one warp takes, many of them, so that each slot in shared
    memory is filled again and again: right, and the same bits each time."""
    T = 20000
    test_norm_in(moe, T, H, BF16, F32)
    g = torch.Generator().manual_seed(H)
    x, y, w = _randn(g, T, H, dtype=BF16), _randn(g, T, H, dtype=BF16), _randn(g, H)
    first = moe.moe_norm_out(x, y, w, next_weight=w, save_rstd=True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, moe.moe_norm_out(x, y, w, next_weight=w, save_rstd=True)))
    back = dict(grad_next=y, out=first[0], next_weight=w, next_rstd=first[3])
    grads = moe.moe_norm_out_backward(x, y, w, first[1], **back)
    for _ in range(5):
        for a, b in zip(grads, moe.moe_norm_out_backward(x, y, w, first[1], **back)):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(7, 96), (5, 33), (1300, 1024), (2000, 2048), (640, 5000), (650, 8192), (640, 8199), (600, 16384)])
@pytest.mark.parametrize("xt,wt,gt", [(BF16, BF16, F32), (F32, BF16, F32), (F32, F32, BF16)])
@pytest.mark.parametrize("gate_kind", ["token", "element"])
def test_norm_out_weights_and_gates(moe, T, H, xt, wt, gt, gate_kind):
    """The other combinations: weights of either type with an offset, and sigmoid
    gates of either type, direct and through shared memory.  The gate's fast
    exponential is within 2 + 1.2 |g| ulp (2^-23), |g| < 15 here: 40 u more,
    and twice that in its slope, inside the tolerance's 320 u beside the row's."""
    g = torch.Generator().manual_seed(T + H)
    x, y = _randn(g, T, H, dtype=xt, std=2.0), _randn(g, T, H, dtype=BF16, std=0.3)
    w, w2 = _randn(g, H, dtype=wt, std=0.2), _randn(g, H, dtype=wt, std=0.2)
    gate = _randn(g, *((T,) if gate_kind == "token" else (T, H)), dtype=gt, std=3.0)
    kw = dict(gate=gate, residual_scale=0.5, weight_offset=1.0)
    out, rstd, nxt, rstd2 = moe.moe_norm_out(x, y, w, next_weight=w2, save_rstd=True, **kw)
    wf, wm, w2f, w2m = 1 + w.double(), 1 + w.double().abs(), 1 + w2.double(), 1 + w2.double().abs()
    s = torch.sigmoid(gate.double()).view(T, -1)
    hat = y.double() * _rms64(y.double(), 1e-6)
    _close(out, 0.5 * x.double() + s * hat * wf, 0.5 * x.double().abs() + s * hat.abs() * wm, "out")
    o = out.double()
    oh = o * _rms64(o, 1e-6)
    _close(nxt, oh * w2f, oh.abs() * w2m, "next")
    dout, dnext = _randn(g, T, H, dtype=xt), _randn(g, T, H, dtype=BF16)
    gx, gy, gg, gw, gw2 = moe.moe_norm_out_backward(dout, y, w, rstd, grad_next=dnext, out=out, next_weight=w2,
                                                    next_rstd=rstd2, **kw)
    dd, dw2, mdd, mw2 = _norm_vjp(out, rstd2, w2f, w2m, dnext)
    d, md = dout.double() + dd, dout.double().abs() + mdd
    _close(gw2, dw2, mw2, "grad_next_weight")
    _close(gx, 0.5 * d, 0.5 * md, "grad_x")
    r = rstd.double()[:, None]
    hat, slope = y.double() * r, s * (1 - s)
    if gate_kind == "element":
        _close(gg, slope * d * hat * wf, slope * md * hat.abs() * wm, "grad_gate")
    else:
        _close(gg, slope[:, 0] * (d * hat * wf).sum(1), slope[:, 0] * (md * hat.abs() * wm).sum(1), "grad_gate")
    e, me = wf * s * d, wm * s * md
    _close(gy, r * e - y.double() * r ** 3 * (e * y.double()).mean(1, keepdim=True),
           r * me + y.double().abs() * r ** 3 * (me * y.double().abs()).mean(1, keepdim=True), "grad_y")
    _close(gw, (s * d * hat).sum(0), (s * md * hat.abs()).sum(0), "grad_weight")
