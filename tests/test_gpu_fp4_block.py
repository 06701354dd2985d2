"""e2m1 codes with a power-of-two scale per 32, against fp64.

Codes and scales are functions of the input with exact quotients, so they have
to equal a numpy restatement bit for bit, and so has the way back.  The products
are compared with fp64 on the same codes: products of codes are exact, and an
fp32 sum that keeps at least 13 bits of the largest term while aligning (what the
tensor cores are known to keep at the least) is within 2^-13 of the terms'
magnitudes' sum, S; scaling and adding K / 32 blocks in fp32 is within (K / 32 +
3) 2^-24 of it, below 2^-15 for K up to 8192.  bf16 output adds half a step,
2^-8 (1 + 2^-8) of the value at the most.  So |error| <= (2^-13 + 2^-15) S +
2^-8 (1 + 2^-8) |value|, element by element.
"""
import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
DEV = "cuda"
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module")
def moe():
    import combine_topk_multihot_gb300 as m
    return m


def quantize_np(v):
    """Codes (one a byte) and scales [rows, blocks] of v [rows, cols] by the rule, in fp64."""
    b = v.astype(np.float64).reshape(v.shape[0], -1, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    e = np.frexp(np.where(bad | (top == 0), 1, top))[1] - 1 - 2            # floor(log2 top) - 2
    e = e + (top >= 7 * np.ldexp(1.0, e))
    e = np.where(bad, 128, np.where(top == 0, -127, np.clip(e, -127, 125)))
    q = np.abs(np.ldexp(np.where(bad[..., None], 0, b), np.where(bad, 0, -e)[..., None]))
    mids = (E2M1[1:8] + E2M1[:7]) / 2
    code = np.zeros(b.shape, np.uint8)
    for i, m in enumerate(mids):                     # midway the even code
        code += (q > m) | ((q == m) & (i % 2 == 1))
    code |= np.where(np.signbit(b) & ~bad[..., None], 8, 0).astype(np.uint8)
    return code.reshape(v.shape), (e + 127).astype(np.uint8)


def pack(code):
    return code[..., ::2] | code[..., 1::2] << 4


def values(codes, scales_rows):
    """fp64 numbers of packed codes [rows, cols / 2] and scales [rows, blocks]."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    s = np.where(scales_rows == 255, np.nan, np.ldexp(1.0, scales_rows.astype(int) - 127))
    return (E2M1[n].reshape(*s.shape, 32) * s[..., None]).reshape(n.shape)


def tiles_np(s):
    """Scales [rows, blocks] in tiles, from the layout's definition."""
    R, B = s.shape
    out = np.zeros((-(-R // 128), -(-B // 4), 32, 4, 4), np.uint8)
    r, b = np.meshgrid(np.arange(R), np.arange(B), indexing="ij")
    out[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = s
    return out


def test_tiles(moe):
    g = torch.Generator().manual_seed(0)
    for R, C in ((1, 32), (5, 160), (130, 96), (384, 1024)):
        s = torch.randint(0, 256, (2, R, C // 32), generator=g, dtype=torch.uint8)
        t = moe.moe_fp4_scale_tiles(s)
        for i in range(2):
            assert np.array_equal(t[i].numpy(), tiles_np(s[i].numpy()))
        assert torch.equal(moe.moe_fp4_scale_rows(t, R, C), s)


def test_refusals_without_a_gpu(moe):
    import ctypes
    from combine_topk_multihot_gb300 import _native as N
    p, odd = ctypes.c_void_p(256), ctypes.c_void_p(264)
    q, d, mm = N.lib.moe_quantize_fp4_block, N.lib.moe_dequantize_fp4_block, N.lib.moe_matmul_fp4_block
    for cols in (0, 16, 33, -32):
        assert q(p, 0, 1, 4, cols, p, p, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
        assert d(p, p, 1, 4, cols, 0, p, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
        assert mm(p, p, 4, p, p, 8, cols, p, None, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(p, 0, 1, 2 ** 31, 32, p, p, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(p, 0, 1, 4, 2 ** 24, p, p, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(p, 0, 2 ** 40, 2 ** 10, 32, p, p, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(p, 7, 1, 4, 32, p, p, None) == N.MOE_ERR_INVALID_ARG
    assert d(p, p, 1, 4, 32, -1, p, None) == N.MOE_ERR_INVALID_ARG
    for bad in (None, odd):
        assert q(bad, 0, 1, 4, 32, p, p, None) == N.MOE_ERR_INVALID_ARG
        assert q(p, 0, 1, 4, 32, bad, p, None) == N.MOE_ERR_INVALID_ARG
        assert q(p, 0, 1, 4, 32, p, bad, None) == N.MOE_ERR_INVALID_ARG
        assert d(bad, p, 1, 4, 32, 0, p, None) == N.MOE_ERR_INVALID_ARG
        assert mm(p, bad, 4, p, p, 8, 32, p, None, None) == N.MOE_ERR_INVALID_ARG
        assert mm(p, p, 4, p, p, 8, 32, bad, None, None) == N.MOE_ERR_INVALID_ARG
    assert mm(p, p, -1, p, p, 8, 32, p, None, None) == N.MOE_ERR_INVALID_ARG
    assert mm(p, p, 4, p, p, 0, 32, p, None, None) == N.MOE_ERR_INVALID_ARG
    assert mm(p, p, 2 ** 31 - 1, p, p, 2 ** 31 - 1, 32, p, None, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert b"tiles" in N.lib.moe_last_error()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no CPU kernel"):
        moe.moe_quantize_fp4_block(x)


def source(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(*shape[:-1], 1, generator=g))
    x[..., 0, :16] = 0
    x[..., -1, 1] = -0.0
    if shape[-2] > 8:
        x[..., 2, :] = 0
        x[..., 3, :] *= 1e-38
        x[..., 4, :] *= 1e-42                      # below the smallest scale's half
        x[..., 5, :] = x[..., 5, :].clamp(-3, 3) * 1e38
        x[..., 6, :] = torch.arange(shape[-1]) % 33 * 0.25 - 4       # every midpoint
        x[..., 7, 5], x[..., 8, -1] = float("nan"), -float("inf")
    return x.to(dtype)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (1, 2048), (7, 128), (130, 288), (33, 4128), (129, 1024), (3, 200, 160),
                                   (2, 3, 40, 96)])
def test_quantize_and_back_bit_exact(moe, shape, dtype):
    src = source(shape, sum(shape), dtype)
    codes, scales = moe.moe_quantize_fp4_block(src.to(DEV))
    back = moe.moe_dequantize_fp4_block(codes, scales)
    back32 = moe.moe_dequantize_fp4_block(codes, scales, torch.float32)
    assert back.dtype is torch.bfloat16 and back.shape == src.shape == back32.shape
    R, C = shape[-2:]
    for i, m in enumerate(src.float().reshape(-1, R, C).numpy()):
        code, e = quantize_np(m)
        assert np.array_equal(codes.cpu().numpy().reshape(-1, R, C // 2)[i], pack(code))
        assert np.array_equal(scales.cpu().numpy().reshape(-1, *scales.shape[-5:])[i], tiles_np(e))
        v = values(pack(code), e)
        assert np.array_equal(back32.cpu().numpy().reshape(-1, R, C)[i].astype(np.float64), v, equal_nan=True)
        assert np.array_equal(back.cpu().float().numpy().reshape(-1, R, C)[i].astype(np.float64), v, equal_nan=True)


@gpu
def test_every_code_and_scale(moe):
    """All 256 bytes of codes under all 256 scales, in both types."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 16, 16).expand(256, 16, 16).reshape(4096, 16).contiguous()
    rows = torch.arange(256, dtype=torch.uint8).view(256, 1).expand(256, 16).reshape(4096, 1).contiguous()
    v = values(codes.numpy(), rows.numpy())
    t = moe.moe_fp4_scale_tiles(rows).to(DEV)
    for dt in (torch.float32, torch.bfloat16):
        got = moe.moe_dequantize_fp4_block(codes.to(DEV), t, dt).float().cpu().numpy()
        with np.errstate(over="ignore"):
            assert np.array_equal(got, v.astype(np.float32), equal_nan=True)


def _bound_check(out, a, b):
    ref, S = a @ b.T, np.abs(a) @ np.abs(b).T
    err = np.abs(out.double().cpu().numpy() - ref)
    lim = (2.0 ** -13 + 2.0 ** -15) * S + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(ref)
    assert (err <= lim).all(), float((err - lim).max())


# few rows by few (up to 8 by 1024: the weight stream), others on the tensor cores:
# every tile width, ragged edges in every dimension, one block of K, K not a
# multiple of 64, 128 or 256
MATMUL = [(8, 1024, 2080), (3, 1023, 96), (8, 1025, 544), (1, 20000, 256), (4000, 192 * 43, 512), (1, 16, 32), (1, 4096, 2048), (7, 100, 160), (8, 4097, 2080), (2, 1, 64), (5, 33, 8192), (9, 64, 32), (9, 1, 64),
          (16, 513, 512), (17, 77, 2080), (64, 1000, 2048), (100, 8, 160), (128, 256, 512), (129, 2048, 1056),
          (300, 4100, 2048), (1000, 384, 4096), (1111, 8192, 256), (2049, 1027, 544), (5000, 4096, 384), (777, 2050, 96)]


@gpu
@pytest.mark.parametrize("M,N,K", MATMUL)
def test_matmul(moe, M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    a = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    b = torch.randn(N, K, generator=g) * 0.05
    b[:, : K // 2] *= 16                           # blocks of unlike scales
    aq, sa = moe.moe_quantize_fp4_block(a.bfloat16().to(DEV))
    bq, sb = moe.moe_quantize_fp4_block(b.to(DEV))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    got = moe.moe_matmul_fp4_block(aq, sa, bq, sb, out=out[:M], status=status)
    assert got.data_ptr() == out.data_ptr() and (out[M] == 7).all() and int(status) == 0
    val = lambda q, s: moe.moe_dequantize_fp4_block(q, s, torch.float32).double().cpu().numpy()  # noqa: E731
    _bound_check(got, val(aq, sa), val(bq, sb))
    again = moe.moe_matmul_fp4_block(aq, sa, bq, sb)
    assert torch.equal(again, got)


@gpu
@pytest.mark.parametrize("M", [3, 40])
def test_matmul_scales(moe, M):
    """Every pair of scales whose product is a bf16 number, and what is too small, too large or NaN."""
    K, N = 64, 256
    aq = torch.full((M, K // 2), 0x22, dtype=torch.uint8)                  # ones
    bq = torch.full((N, K // 2), 0x22, dtype=torch.uint8)
    for ea in (0, 1, 100, 127, 200, 254, 255):
        sa = torch.full((M, K // 32), ea, dtype=torch.uint8)
        sb = torch.arange(N, dtype=torch.uint8).view(N, 1).expand(N, K // 32).contiguous()
        out = moe.moe_matmul_fp4_block(aq.to(DEV), moe.moe_fp4_scale_tiles(sa).to(DEV), bq.to(DEV),
                                       moe.moe_fp4_scale_tiles(sb).to(DEV)).double().cpu().numpy()
        e = ea + np.arange(N) - 254 + 6                                     # 64 ones
        nan = (np.arange(N) == 255) | (ea == 255)
        normal = (e >= -120) & (e <= 127) & ~nan
        assert np.isnan(out[:, nan]).all()
        assert (out[:, normal] == np.ldexp(1.0, e[normal])).all()
        assert np.isinf(out[:, (e > 127) & ~nan]).all()
        assert (np.abs(out[:, (e < -120) & ~nan]) <= 2.0 ** -120).all()


@gpu
def test_no_rows_and_refusals(moe):
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    c, s = moe.moe_quantize_fp4_block(torch.zeros(0, 64, device=DEV))
    assert c.shape == (0, 32) and s.shape == (0, 1, 32, 4, 4)
    assert moe.moe_dequantize_fp4_block(c, s).shape == (0, 64)
    bq, sb = moe.moe_quantize_fp4_block(torch.ones(5, 64, device=DEV))
    assert moe.moe_matmul_fp4_block(c, s, bq, sb).shape == (0, 5)
    for bad in (torch.zeros(4, 40, device=DEV), torch.zeros(64, device=DEV), torch.zeros(4, 0, device=DEV)):
        with pytest.raises(ValueError):
            moe.moe_quantize_fp4_block(bad)
    with pytest.raises(TypeError):
        moe.moe_quantize_fp4_block(torch.zeros(4, 64, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_quantize_fp4_block(torch.zeros(64, 64, device=DEV).t())
    with pytest.raises(TypeError):
        moe.moe_dequantize_fp4_block(bq, sb, torch.float16)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_dequantize_fp4_block(bq, sb[:, :, :, :, :2].contiguous())
    with pytest.raises(ValueError, match="shape"):
        moe.moe_matmul_fp4_block(bq, sb, z(5, 16), z(1, 1, 32, 4, 4))
    with pytest.raises(moe.MoEError):                                       # codes that do not start on 16 bytes
        moe.moe_dequantize_fp4_block(z(5 * 32 + 8)[8:].view(5, 32), sb)


@gpu
def test_on_another_stream_and_captured(moe):
    x = torch.randn(40, 512, device=DEV)
    bq, sb = moe.moe_quantize_fp4_block(torch.randn(96, 512, device=DEV))
    want = [moe.moe_matmul_fp4_block(*moe.moe_quantize_fp4_block(x[:m]), bq, sb) for m in (5, 40)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for m in (5, 40):
        a, sa = moe.moe_quantize_fp4_block(x[:m], stream=side)
        got.append(moe.moe_matmul_fp4_block(a, sa, bq, sb, stream=side))
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [moe.moe_matmul_fp4_block(*moe.moe_quantize_fp4_block(x[:m]), bq, sb) for m in (5, 40)]
    x.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, -2 * w) for g, w in zip(held, want))


def test_sizes_past_32_bits_are_refused_without_a_gpu(moe, monkeypatch):
    """K of 2^31 - 32, which rounded up passes 32 bits, and sizes that would cross to the library without their upper bits."""
    import ctypes
    from combine_topk_multihot_gb300 import _native as N, block
    p = ctypes.c_void_p(256)
    for K in (2 ** 29 + 32, 2 ** 30, 2 ** 31 - 256, 2 ** 31 - 32):
        for M in (1, 9, 300):
            assert N.lib.moe_matmul_fp4_block(p, p, M, p, p, 8, K, p, None, None) == N.MOE_ERR_UNSUPPORTED_SHAPE
            assert b"2^29" in N.lib.moe_last_error()
    monkeypatch.setattr(block, "_on_gpu", lambda t, name: t.device)
    big = lambda *s, dt=torch.uint8: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="below 2\\^31"):
        moe.moe_quantize_fp4_block(big(1, 2 ** 32 + 32, dt=torch.bfloat16))
    with pytest.raises(ValueError, match="below 2\\^31"):
        moe.moe_dequantize_fp4_block(big(1, 2 ** 31 + 16), big(1, 2 ** 25 + 1, 32, 4, 4))
    small, scales = big(8, 16), big(1, 1, 32, 4, 4)
    for a, b in ((big(1, 2 ** 31 + 16), small), (big(2 ** 32 + 1, 16), small), (small, big(2 ** 32 + 1, 16))):
        with pytest.raises(ValueError, match="below 2\\^31"):
            moe.moe_matmul_fp4_block(a, scales, b, scales)


def test_scale_rows_that_the_tiles_do_not_hold(moe):
    t = torch.arange(2 * 512, dtype=torch.int32).to(torch.uint8).view(1, 2, 32, 4, 4)
    assert moe.moe_fp4_scale_rows(t, 128, 256).shape == (128, 8) and moe.moe_fp4_scale_rows(t, 0, 0).shape == (0, 0)
    for rows, cols in ((129, 256), (128, 288), (-1, 32), (5, 40), (5, -32)):
        with pytest.raises(ValueError, match="hold no"):
            moe.moe_fp4_scale_rows(t, rows, cols)
    for bad in (t[0, 0], t.view(1, 2, 32, 2, 8), t.view(2, 512)):
        with pytest.raises(ValueError, match="tiles must be"):
            moe.moe_fp4_scale_rows(bad, 1, 32)
