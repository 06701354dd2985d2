"""A block-scaled product or a norm whose operands stop arriving ends by its own bounded
waits (about 2 s), says so in the status word if it has one, and leaves NaN wherever it did
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
    assert moe._native.lib.moe_selftest_norm_rows(-2) == moe._native.MOE_ERR_INVALID_ARG


@contextlib.contextmanager
def _rows(moe, n):
    lib = moe._native.lib
    assert lib.moe_selftest_norm_rows(n) == moe._native.MOE_OK
    try:
        yield
    finally:
        assert lib.moe_selftest_norm_rows(-1) == moe._native.MOE_OK


def _call(moe, rows, fn):
    """fn's outputs with `rows` rows arriving.  The allocator's blocks hold numbers before, so
    that what is not written cannot look like NaN."""
    torch.cuda.synchronize()
    held = [torch.zeros(n, device=DEV) for n in (1 << 12, 1 << 14, 1 << 20, 1 << 23, 1 << 23, 1 << 23)]
    del held
    with _rows(moe, rows):
        got = fn()
    torch.cuda.synchronize()
    return got


# one warp a row, several groups a CTA, one; fp32 and bf16 streams
@pytest.mark.parametrize("T,H,xt,gate_kind,gt", [
    (9000, 264, torch.bfloat16, "token", torch.float32), (3000, 1024, torch.float32, "token", torch.bfloat16),
    (1300, 4096, torch.bfloat16, "element", torch.bfloat16), (700, 8192, torch.float32, "element", torch.float32)])
def test_norms(moe, T, H, xt, gate_kind, gt):
    g = torch.Generator().manual_seed(H)
    rnd = lambda *s, dt=torch.float32: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
    x, y, dn, w = rnd(T, H, dt=xt), rnd(T, H, dt=torch.bfloat16), rnd(T, H, dt=torch.bfloat16), rnd(H)
    gate = rnd(*((T,) if gate_kind == "token" else (T, H)), dt=gt)
    out, rstd, nxt, rstd2 = moe.moe_norm_out(x, y, w, gate=gate, next_weight=w, save_rstd=True)
    forms = [
        lambda: moe.moe_norm_in(x, w, save_rstd=True),
        lambda: moe.moe_norm_out(x, y, w, gate=gate, next_weight=w, save_rstd=True),
        lambda: moe.moe_norm_in_backward(dn, x, w, rstd2),
        lambda: moe.moe_norm_out_backward(x, y, w, rstd, gate=gate, grad_next=dn, out=out, next_weight=w, next_rstd=rstd2),
    ]
    if gate_kind == "token":        # (each wait takes 2 s: not every form at every size)
        forms.append(lambda: moe.moe_norm_out_backward(x, y, w, rstd))
    else:
        forms = forms[1::2]
    for fn in forms:
        whole = [t for t in fn() if t is not None]
        for t in (t for t in _call(moe, 0, fn) if t is not None):
            assert t.isnan().all()
        for a, b in zip(whole, (t for t in fn() if t is not None)):
            assert torch.equal(a, b)


def test_norm_rows_that_arrived_stand(moe):
    T, H = 9000, 512
    x, w = torch.randn(T, H, device=DEV).bfloat16(), torch.ones(H, device=DEV)
    whole = moe.moe_norm_in(x, w, save_rstd=True)
    part = _call(moe, 4000, lambda: moe.moe_norm_in(x, w, save_rstd=True))
    for a, b in zip(whole, part):
        assert b[4000:].isnan().all()
        there = ~b[:4000].isnan()
        assert torch.equal(a[:4000][there], b[:4000][there]) and there.any()
