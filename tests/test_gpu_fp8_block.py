"""e4m3 products with a scale per block of 128, against fp64.

Codes and scales are functions of the bf16 input with IEEE operations, so they
have to equal a numpy restatement bit for bit.  The products are compared with
fp64 on the same codes: products of codes are exact, and an fp32 sum of n terms
that keeps at least 13 bits of the largest term while aligning (what the tensor
cores are known to keep at the least) is within 2^-13 of the terms'
magnitudes' sum, S; the blocks' fp32 scaling and adding is within (K / 128 + 3)
2^-24 of it.  bf16 output adds 2^-8 (1 + 2^-8) of the value.  So
|error| <= (2^-13 + 2^-16) S + 2^-8 (1 + 2^-8) |value|, element by element.

The experts' second product takes codes of h that depend on roundings of the
first: one code may move to its neighbour, at most 1/8 of its size (a step of
e4m3; 2^-9 in units of the scale among the smallest).  The oracle's h is fp64;
moved codes are those whose quotient lies within its error of a midpoint, a few
in 10^4.  y is held to the bf16 GEMM tolerances of the other expert tests
(max |err| <= 2e-2, relative L2 <= 5e-3).
"""
import numpy as np
import pytest
import torch

import oracle as O
from tests._util import assert_gemm_close, bits, random_routing

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_multihot_gb300 as m
    return m


def _quantize_np(v, block_rows):
    """Codes and scales of v [rows, cols] fp32 by the rule."""
    f = np.float32
    R, C = v.shape
    pr, pc = -R % block_rows, -C % 128
    b = np.pad(v, ((0, pr), (0, pc))).reshape((R + pr) // block_rows, block_rows, (C + pc) // 128, 128)
    top = np.abs(b).max((1, 3))
    scale = np.where(top == 0, f(1), np.maximum(top / f(448), f(2.0 ** -126)))
    q = (b / scale[:, None, :, None]).reshape(R + pr, C + pc)[:R, :C]
    codes = torch.from_numpy(np.ascontiguousarray(q)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.numpy(), scale


def _values(codes, scales, block_rows):
    """The fp64 numbers that codes [rows, cols] on the GPU stand for."""
    R, C = codes.shape
    s = scales.double().repeat_interleave(block_rows, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return codes.view(torch.float8_e4m3fn).double() * s


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (1, 2048), (7, 128), (130, 272), (33, 4112), (129, 1024), (3, 200, 144)])
def test_quantize_bit_exact(moe, shape, block_rows):
    g = torch.Generator().manual_seed(sum(shape))
    src = (torch.randn(*shape, generator=g) * torch.exp(3 * torch.randn(*shape[:-1], 1, generator=g))).bfloat16()
    src[..., 0, :16] = 0
    if shape[-2] > 2:
        src[..., 2, :] = 0
    if shape[-2] > 4:
        src[..., 4, :] *= 1e-38                   # subnormal scales are held at 2^-126
    codes, scales = moe.moe_quantize_fp8_block(src.to(DEV), block_rows)
    lead = src.reshape(-1, *shape[-2:]).float().numpy()
    for i, m in enumerate(lead):
        c, s = _quantize_np(m, block_rows)
        assert np.array_equal(codes.cpu().numpy().reshape(lead.shape)[i], c)
        assert np.array_equal(scales.cpu().numpy().reshape(-1, *s.shape)[i], s)


def test_quantize_division_rounds_as_ieee(moe):
    """Every pair of a bf16 significand and a block maximum's significand (128 x
    128, in all binades that matter), so that each quotient midway between two
    codes is met: equal to codes from an IEEE division, bit for bit."""
    top = torch.arange(128, 256, dtype=torch.float32).view(128, 1, 1)          # a row each
    sig = torch.arange(128, 256, dtype=torch.float32).view(1, 1, 128)
    # halves of 64 significands: the block's first value is its maximum
    for e in range(0, 20):
        v = (sig * 2.0 ** -e).clamp(max=1e30).expand(128, 2, 128).clone()
        v[v > top] *= 0.5
        v[:, 0, 0] = top[:, 0, 0]
        v[:, 1, 1] = top[:, 0, 0]
        for scale in (2.0 ** -20, 2.0 ** -110, 2.0 ** 60):
            src = (v * scale).reshape(128, 256).bfloat16()
            codes, scales = moe.moe_quantize_fp8_block(src.to(DEV))
            c, s = _quantize_np(src.float().numpy(), 1)
            assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s), (e, scale)


def test_quantize_nonfinite(moe):
    src = torch.ones(3, 384, dtype=torch.bfloat16, device=DEV)
    src[0, 5], src[1, 200] = float("nan"), float("inf")
    _, s = moe.moe_quantize_fp8_block(src)
    finite = torch.isfinite(s).cpu().tolist()
    assert finite == [[False, True, True], [True, False, True], [True, True, True]]
    a, sa = moe.moe_quantize_fp8_block(torch.cat([src, src[2:].repeat(61, 1)]))
    b, sb = moe.moe_quantize_fp8_block(torch.ones(64, 384, dtype=torch.bfloat16, device=DEV), 128)
    for m in (3, 64):
        out = moe.moe_matmul_fp8_block(a[:m], sa[:m], b, sb)
        assert not torch.isfinite(out[:2]).any() and torch.isfinite(out[2:]).all()


# few rows (1 to 8: the weight stream), more on the tensor cores: the three tile
# widths, ragged edges in every dimension, one K block, K not a multiple of 128
MATMUL = [(1, 16, 16), (1, 4096, 2048), (7, 100, 128), (8, 64, 1024), (9, 129, 400), (16, 513, 512), (17, 77, 2064),
          (32, 2048, 768), (33, 64, 128), (64, 1000, 2048), (100, 8, 144), (128, 256, 512), (129, 2048, 1040),
          (300, 4100, 2048), (1000, 384, 4096), (1111, 8192, 256), (2049, 1027, 512), (5000, 4096, 384),
          (5001, 4099, 384), (777, 2050, 640)]


@pytest.mark.parametrize("M,N,K", MATMUL)
def test_matmul(moe, M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    a = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).bfloat16().to(DEV)
    b = (torch.randn(N, K, generator=g) * 0.05).bfloat16().to(DEV)
    b[:, : K // 2] *= 16                          # blocks of unlike scales
    aq, sa = moe.moe_quantize_fp8_block(a)
    bq, sb = moe.moe_quantize_fp8_block(b, 128)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    moe.moe_matmul_fp8_block(aq, sa, bq, sb, out=out, status=status)
    assert int(status) == 0
    a64, b64 = _values(aq, sa, 1), _values(bq, sb, 128)
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    tol = (2.0 ** -13 + 2.0 ** -16) * mag + 2.0 ** -8 * (1 + 2.0 ** -8) * ref.abs()
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    again = moe.moe_matmul_fp8_block(aq, sa, bq, sb)
    assert torch.equal(out, again)


def _experts_ref(xd, counts, offsets, w, W1, s1, W2, s2, I):
    """y in fp64 from the rows of x_disp, with the two quantisations."""
    y = torch.zeros(xd.shape, dtype=torch.float64)
    for e, n in enumerate(counts):
        if not n:
            continue
        r = slice(offsets[e], offsets[e] + n)
        q, s = _quantize_np(xd[r].float().numpy(), 1)
        x = _values(torch.from_numpy(q), torch.from_numpy(s), 1)
        gu = x @ _values(W1[e], s1[e], 128).T
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        q, s = _quantize_np(h.float().numpy(), 1)
        o = _values(torch.from_numpy(q), torch.from_numpy(s), 1) @ _values(W2[e], s2[e], 128).T
        y[r] = o * w[r].double()[:, None]
    return y


@pytest.mark.parametrize("T,H,E,K,I,P,drop", [
    (1, 256, 8, 2, 128, 1, 0.0), (1, 2048, 128, 8, 768, 1, 0.0), (5, 512, 4, 4, 384, 16, 0.3),
    (13, 256, 8, 2, 256, 1, 0.1), (32, 768, 8, 3, 128, 8, 0.0), (33, 256, 8, 2, 128, 1, 0.0),
    (200, 512, 16, 4, 256, 128, 0.1), (700, 1024, 8, 2, 640, 1, 0.0), (300, 256, 1024, 2, 128, 1, 0.0),
    (64, 256, 8, 1, 128, 4, 1.0),   # every slot dropped: no rows at all
    (40, 256, 4, 1, 128, 1, 0.0),
    (8, 1024, 8, 4, 256, 4, 0.1), (9, 1024, 8, 4, 256, 4, 0.1),   # the two sides of the rule on rows
])
def test_experts(moe, T, H, E, K, I, P, drop):
    idx, p = random_routing(T, E, K, seed=T + H, drop=drop)
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).bfloat16()
    W1 = (torch.randn(E, 2 * I, H, generator=g) * 0.05).bfloat16().to(DEV)
    W2 = (torch.randn(E, H, I, generator=g) * 0.05).bfloat16().to(DEV)
    q1, s1 = moe.moe_quantize_fp8_block(W1, 128)
    q2, s2 = moe.moe_quantize_fp8_block(W2, 128)
    C = moe.worst_case_rows(T, E, K, P)
    L = moe.Layout(T, E, K, P, C, device=DEV)
    xd, _, _ = moe.moe_dispatch_topk(x.to(DEV), idx.to(DEV), p.to(DEV), L, host_sync=False)
    y = torch.full((C, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2, out=y)
    torch.cuda.synchronize()
    assert int(L.status) == 0
    counts, offsets = L.tokens_per_expert.cpu().tolist(), L.offsets.cpu().tolist()
    ref = _experts_ref(xd.cpu(), counts, offsets, L.row_weight.cpu(), q1.cpu(), s1.cpu(), q2.cpu(), s2.cpu(), I)
    valid = (L.row_token >= 0).cpu()
    assert int(valid.sum()) == sum(counts)
    yc = y.cpu()
    assert yc[~valid].isnan().all()               # pad and spare rows are not touched
    if valid.any():
        assert_gemm_close(bits(yc[valid]), O.f64_to_bf16_bits(ref[valid].numpy()), "y")


def test_experts_captured_and_repeated(moe):
    T, H, E, K, I, P = 48, 512, 8, 2, 256, 1
    g = torch.Generator().manual_seed(1)
    idx, p = random_routing(T, E, K, seed=1)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    q1, s1 = moe.moe_quantize_fp8_block((torch.randn(E, 2 * I, H, generator=g) * 0.05).bfloat16().to(DEV), 128)
    q2, s2 = moe.moe_quantize_fp8_block((torch.randn(E, H, I, generator=g) * 0.05).bfloat16().to(DEV), 128)
    L = moe.Layout(T, E, K, P, T * K, device=DEV)
    xd, _, _ = moe.moe_dispatch_topk(x, idx.to(DEV), p.to(DEV), L, host_sync=False)
    first = moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe.moe_grouped_experts_fp8_block(xd, L, q1, s1, q2, s2)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)


def test_refusals(moe):
    a = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    aq, sa = moe.moe_quantize_fp8_block(a)
    bq, sb = moe.moe_quantize_fp8_block(torch.zeros(128, 256, dtype=torch.bfloat16, device=DEV), 128)
    with pytest.raises(TypeError, match="src must be"):
        moe.moe_quantize_fp8_block(a.float())
    with pytest.raises(ValueError, match="block_rows"):
        moe.moe_quantize_fp8_block(a, 64)
    with pytest.raises(moe.MoEError, match="multiple of 16"):
        moe.moe_quantize_fp8_block(a[:, :8].contiguous())
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_quantize_fp8_block(a.cpu())
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_quantize_fp8_block(a[:, ::2])
    with pytest.raises(ValueError, match="b_q must have shape"):
        moe.moe_matmul_fp8_block(aq, sa, bq[:, :128].contiguous(), sb)
    with pytest.raises(ValueError, match="b_scale"):
        moe.moe_matmul_fp8_block(aq, sa, bq, sb[:, :1].contiguous())
    with pytest.raises(TypeError, match="a_q"):
        moe.moe_matmul_fp8_block(a, sa, bq, sb)
    L = moe.Layout(4, 8, 2, 1, 8, device=DEV)
    xd = torch.zeros(8, 256, dtype=torch.bfloat16, device=DEV)
    w1, s1 = moe.moe_quantize_fp8_block(torch.zeros(8, 256, 256, dtype=torch.bfloat16, device=DEV), 128)
    w2, s2 = moe.moe_quantize_fp8_block(torch.zeros(8, 256, 128, dtype=torch.bfloat16, device=DEV), 128)
    with pytest.raises(ValueError, match="x_disp"):
        moe.moe_grouped_experts_fp8_block(xd[:4], L, w1, s1, w2, s2)
    with pytest.raises(ValueError, match="W2_scale"):
        moe.moe_grouped_experts_fp8_block(xd, L, w1, s1, w2, s1)
    empty = moe.moe_matmul_fp8_block(aq[:0], sa[:0], bq, sb)
    assert empty.shape == (0, 128)


@pytest.mark.parametrize("N,K", [(100, 128), (1027, 2064), (4096, 512)])
def test_few_rows_as_among_many(moe, N, K):
    """A row's product is the same, to its rounding, whether it comes alone (the
    weight stream), among 8, or in a tile of 128: each is within the bound
    above of fp64, so two are within twice that."""
    g = torch.Generator().manual_seed(N)
    aq, sa = moe.moe_quantize_fp8_block(torch.randn(130, K, generator=g).bfloat16().to(DEV))
    bq, sb = moe.moe_quantize_fp8_block(torch.randn(N, K, generator=g).bfloat16().to(DEV), 128)
    whole = moe.moe_matmul_fp8_block(aq, sa, bq, sb)
    mag = _values(aq, sa, 1).abs() @ _values(bq, sb, 128).abs().T
    for m in (1, 2, 7, 8, 9, 16, 64, 128):
        part = moe.moe_matmul_fp8_block(aq[:m], sa[:m], bq, sb)
        tol = 2 * ((2.0 ** -13 + 2.0 ** -16) * mag[:m] + 2.0 ** -8 * (1 + 2.0 ** -8) * whole[:m].double().abs() * (1 + 2.0 ** -7))
        assert ((part.double() - whole[:m].double()).abs() <= tol).all(), m
