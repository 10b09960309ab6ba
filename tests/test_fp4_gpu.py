"""4-bit linears on the GPU: codes and scales against the rule, products and chains against 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
import fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])


def ok():
    torch.cuda.synchronize()
    assert sgq.sgq_device_status() == 0


def randn(*shape, seed=0, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def one(t):
    return torch.full((1,), t, dtype=torch.float32, device=DEV)


def check_quant(x, fmt, t=None, out=None):
    """quant_fp4 of x against the rule, bit for bit, padding of the scale tiles included."""
    ts = None if t is None else one(t)
    q, s = sgq.quant_fp4(x, fmt, tensor_scale=ts, **(out or {}))
    ok()
    nib, byte = ref.quantise(x.float().cpu().numpy(), fmt, 1.0 if t is None else np.float32(t))
    assert np.array_equal(ref.unpack(q), nib)
    M, K = x.shape
    G = s.shape[1] * 4
    got = ref.from_tiles(s, M, G)
    assert np.array_equal(got[:, :K // ref.GROUP[fmt]], byte)
    assert (got[:, K // ref.GROUP[fmt]:] == 0).all()
    return q, s


# ---------------------------------------------------------------- quantisation

@BOTH
@TYPES
@pytest.mark.parametrize("M,K", [(1, 32), (1, 7168), (3, 96), (127, 160), (128, 512), (130, 544), (33, 1056), (700, 4064)])
def test_quant_is_the_rule(fmt, dtype, M, K):
    check_quant(randn(M, K, seed=M + K, dtype=dtype, std=3.0), fmt, 0.0371 if fmt == "nvfp4" else None)


@pytest.mark.parametrize("t", [None, 1e-4, 3e3, 0.037109375, 1e-30, 1e30])
def test_nvfp4_scales_of_any_size(t):
    """Groups whose scale is below E4M3's smallest value, or above its largest (values saturate), or between."""
    x = randn(64, 512, seed=5) * torch.logspace(-12, 12, 64, base=2.0, device=DEV)[:, None].bfloat16()
    check_quant(x, "nvfp4", t)


@BOTH
@TYPES
def test_quant_values_next_to_borders(fmt, dtype):
    """Every 16-bit pattern of the type that is finite, each in groups with other values; ties, signed zeros, subnormals."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(dtype)
    x = x[torch.isfinite(x)]
    top = 1e30 if dtype == torch.bfloat16 else 6e4
    x = x[x.abs().float() < top]
    g = torch.Generator("cpu").manual_seed(1)
    for order in (torch.arange(x.numel()), torch.randperm(x.numel(), generator=g)):
        y = x[order]
        y = y[:y.numel() // 512 * 512].view(-1, 512).to(DEV)
        check_quant(y, fmt, 0.5 if fmt == "nvfp4" else None)
    # multiples of a half at scale 1: ties of every level, both signs
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, 4.0, 1.0, 0.5, 2.0, 3.0, 1.5, 5.5])
    y = torch.cat([ties, -ties]).repeat(3, 2).to(dtype).to(DEV)
    check_quant(y, fmt, 1.0 if fmt == "nvfp4" else None)


@BOTH
@TYPES
def test_quant_of_groups_that_are_not_finite(fmt, dtype):
    x = randn(5, 256, seed=2, dtype=dtype)
    x[0, 3], x[1, 40], x[2, 255], x[3, 64:96] = float("nan"), float("inf"), -float("inf"), float("nan")
    q, s = check_quant(x, fmt)
    v = sgq.dequant_fp4(q, s, fmt, dtype=dtype)
    bad = torch.isnan(v).view(5, -1, ref.GROUP[fmt])
    want = (~torch.isfinite(x)).view(5, -1, ref.GROUP[fmt]).any(-1, keepdim=True).expand_as(bad)
    assert torch.equal(bad, want)


@BOTH
@pytest.mark.parametrize("shift", [0, 8, 16, 24])
@pytest.mark.parametrize("K", [512, 1024, 1056])
def test_quant_of_rows_that_start_anywhere(fmt, shift, K):
    """Rows on 16 bytes or on 32, whole spans of 512 or not, even and odd numbers of rows."""
    for M in (1, 2, 301, 2000):
        wide = randn(M * (K + 40) + 64, seed=shift)
        for step in (K + 8, K + 16):
            check_quant(torch.as_strided(wide, (M, K), (step, 1), shift), fmt)


@BOTH
def test_quant_of_rows_apart_into_given_outputs(fmt):
    """x is a part of wider rows; outputs lie between guards that stay."""
    wide = randn(257, 2048 + 64, seed=3)
    x = wide[:, 32:32 + 1120]
    M, K = x.shape
    T = -(-K // (128 if fmt == "mxfp4" else 64))
    q = torch.full((M * K // 2 + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((3 * T * 512 + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    xq, xs = q[32:-32].view(M, K // 2), s[32:-32].view(3, T, 512)
    check_quant(x, fmt, out=dict(xq=xq, xs=xs))
    for guard in (q[:32], q[-32:], s[:32], s[-32:]):
        assert (guard == 0xA5).all()
    pad = ref.from_tiles(xs, 384, T * 4)[M:]
    assert (pad == 0xA5).all()           # rows past the last one are left as they were


@BOTH
@TYPES
@pytest.mark.parametrize("M,K", [(1, 64), (37, 1056), (130, 512)])
def test_quant_silu_mul(fmt, dtype, M, K):
    """silu(g) u is within 2^-18 of its value, its codes and scales follow from that."""
    x = randn(M, 2 * K, seed=K, dtype=dtype, std=2.0)
    x[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 88.0, -88.0, 5.0, -5.0])
    t = 0.011
    q, s = sgq.quant_fp4(x, fmt, tensor_scale=one(t) if fmt == "nvfp4" else None, silu_mul=True)
    ok()
    g, u = ref.f64(x)[:, :K], ref.f64(x)[:, K:]
    y = g / (1 + np.exp(-g)) * u
    ref.check_codes(ref.unpack(q), ref.from_tiles(s, M, K // ref.GROUP[fmt]), y, fmt, np.float32(t), 2.0 ** -18, f"{fmt} {M}x{K}")


@BOTH
def test_quant_silu_mul_of_gates_far_below_zero(fmt):
    """silu(g) is 2^-120 and less here, times u up to bf16's largest; to where exp(-g) leaves fp32."""
    K = 512
    g = -torch.linspace(80, 88.5, 9).bfloat16()[:, None].expand(9, K)
    u = (torch.rand(9, K, generator=torch.Generator().manual_seed(3)) + 0.5).mul(2.0 ** 126).bfloat16()
    q, s = sgq.quant_fp4(torch.cat([g, u], 1).to(DEV), fmt, silu_mul=True)
    ok()
    g, u = ref.f64(g), ref.f64(u)
    y = g / (1 + np.exp(-g)) * u
    # the exponent, 127 and less, is off by 2^-18 (its rounding) and 127 2^-26 (log2 e's): 1.5 2^-18 times ln 2
    ref.check_codes(ref.unpack(q), ref.from_tiles(s, 9, K // ref.GROUP[fmt]), y, fmt, np.float32(1), 2.0 ** -17, fmt)


@pytest.mark.parametrize("t", [2.0 ** -126, 2.0 ** -131, 2.0 ** -149])
def test_quant_under_the_smallest_tensor_scales(t):
    """Divisors below fp32's normal numbers, whose reciprocals are infinite; groups of zeros.  silu(32) is 32 within 2^-46."""
    K = 1056
    u = (randn(5, K, seed=1).float().cpu() * 2.0 ** torch.linspace(-133, -122, K // 16).repeat_interleave(16)).bfloat16()
    u[:, 16:32] = 0
    check_quant(u.to(DEV), "nvfp4", t)
    q, s = sgq.quant_fp4(torch.cat([torch.full_like(u, 32.0), u], 1).to(DEV), "nvfp4", tensor_scale=one(t), silu_mul=True)
    ok()
    ref.check_codes(ref.unpack(q), ref.from_tiles(s, 5, K // 16), 32 * ref.f64(u), "nvfp4", np.float32(t), 2.0 ** -17)
    assert ((ref.unpack(q) & 7)[:, 16:32] == 0).all()


@BOTH
@TYPES
@pytest.mark.parametrize("M,K", [(1, 32), (129, 544), (300, 1568)])
def test_dequant_is_the_rounded_value(fmt, dtype, M, K):
    """All codes and all scale bytes (but MXFP4's that leave the type), rounded once."""
    rng = np.random.default_rng(M)
    nib = rng.integers(0, 16, (M, K)).astype(np.uint8)
    span = (112, 140) if fmt == "mxfp4" else (0, 127)
    byte = rng.integers(*span, (M, K // ref.GROUP[fmt])).astype(np.uint8)
    t = 1.0 if fmt == "mxfp4" else 0.0137
    xq, xs = torch.from_numpy(ref.pack(nib)).to(DEV), torch.from_numpy(ref.to_tiles(byte, 0xFF)).to(DEV)
    v = sgq.dequant_fp4(xq, xs, fmt, tensor_scale=one(t) if fmt == "nvfp4" else None, dtype=dtype)
    ok()
    want = torch.from_numpy(ref.values(nib, byte, fmt, t).astype(np.float32)).to(dtype)
    assert torch.equal(v.cpu(), want)
    out = torch.empty(M * K + 8, dtype=dtype, device=DEV)[8:].view(M, K)     # 16-byte, not 32-byte aligned
    assert torch.equal(sgq.dequant_fp4(xq, xs, fmt, tensor_scale=one(t) if fmt == "nvfp4" else None, out=out).cpu(), want)


# ---------------------------------------------------------------- products

def form(rows, K, fmt, seed, exact):
    """A random tensor in the 4-bit form (numpy nibbles and bytes).  exact: scales whose products' sums are exact in fp32."""
    rng = np.random.default_rng(seed)
    nib = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    if fmt == "mxfp4":
        byte = rng.integers(126, 129, (rows, K // 32)) if exact else rng.integers(115, 131, (rows, K // 32))
    else:   # E4M3 bytes of 0.5, 1, 1.5, 2 (0x30, 0x38, 0x3C, 0x40)
        byte = rng.choice([0x30, 0x38, 0x3C, 0x40], (rows, K // 16)) if exact else rng.integers(1, 127, (rows, K // 16))
    return nib, byte.astype(np.uint8)


def on_gpu(nib, byte, fill=0xFF):
    """Scale rows past the last one hold NaN."""
    return torch.from_numpy(ref.pack(nib)).to(DEV), torch.from_numpy(ref.to_tiles(byte, fill)).to(DEV)


def guarded(M, N, dtype):
    buf = torch.full((M * N + 64,), 7.0, dtype=dtype, device=DEV)
    return buf, buf[32:-32].view(M, N)


#: Sizes where the kernels' tiles, splits and rings begin and end: token tiles of 16, 32, 64, 128, pairs of 256 and 512;
#: weight tiles of 128 and 192; stages of 256 along K, MMAs of 64; splits of 1 to 8.
SIZES = [(1, 8, 32), (1, 128, 64), (2, 136, 96), (16, 1536, 7168), (17, 256, 288), (31, 120, 2048), (33, 264, 544), (64, 7168, 2048),
         (65, 128, 256), (65, 1536, 7168), (100, 200, 4096), (128, 512, 8224), (129, 24576, 1536), (257, 1000, 320), (301, 1536, 7168),
         (513, 192, 64), (512, 7168, 2048), (777, 8, 2080), (1024, 7168, 1024), (1025, 1544, 7168), (2049, 4096, 224), (2600, 7168, 512)]


@BOTH
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_is_exact_where_fp32_is(fmt, M, N, K):
    """Sums of multiples of 1/16 below 2^20: every order of fp32 additions gives the exact value, D is it, rounded once."""
    a, w = form(M, K, fmt, M + K, True), form(N, K, fmt, N + K, True)
    dtype = torch.bfloat16 if (M + N) % 16 else torch.float16
    scale = 1.0 if dtype == torch.bfloat16 else 2.0 ** -6
    t = (None, None) if fmt == "mxfp4" else (one(0.5), one(2.0 * scale))
    buf, out = guarded(M, N, dtype)
    if fmt == "mxfp4" and dtype == torch.float16:
        w = w[0], (w[1] - 6).astype(np.uint8)
    d = sgq.fp4_gemm(*on_gpu(*a), *on_gpu(*w), fmt, x_scale=t[0], w_scale=t[1], out=out)
    ok()
    av, wv = (torch.from_numpy(ref.values(*v, fmt)).to(DEV) for v in (a, w))
    want = av @ wv.T if fmt == "mxfp4" else av @ wv.T * scale
    assert torch.equal(d, want.float().to(dtype))
    assert (buf[:32] == 7).all() and (buf[-32:] == 7).all()


@BOTH
@TYPES
@pytest.mark.parametrize("M,N,K", [(1, 7168, 2048), (48, 1536, 7168), (200, 2048, 1568), (600, 1000, 4096), (1300, 2048, 7168)])
def test_product_of_quantised_values(fmt, dtype, M, N, K):
    """Scales of any size, values as quantisation gives them, against 64 bits."""
    x, w = randn(M, K, seed=1, dtype=dtype), randn(N, K, seed=2, dtype=dtype, std=0.02)
    tx, tw = (None, None) if fmt == "mxfp4" else (sgq.fp4_tensor_scale(x), sgq.fp4_tensor_scale(w))
    (xq, xs), (wq, ws) = sgq.quant_fp4(x, fmt, tensor_scale=tx), sgq.quant_fp4(w, fmt, tensor_scale=tw)
    d = sgq.fp4_gemm(xq, xs, wq, ws, fmt, x_scale=tx, w_scale=tw, dtype=dtype)
    ok()
    rows = np.unique(np.concatenate([np.arange(0, M, 37), [M - 1]]))
    a = ref.values(ref.unpack(xq), ref.from_tiles(xs, M, K // ref.GROUP[fmt]), fmt)[rows]
    b = ref.values(ref.unpack(wq), ref.from_tiles(ws, N, K // ref.GROUP[fmt]), fmt)
    alpha = 1.0 if tx is None else float(np.float32(tx.item()) * np.float32(tw.item()))
    ref.check_product(d[torch.from_numpy(rows).to(DEV)], a, b, alpha, dtype, f"{fmt} {M}x{N}x{K}")


@BOTH
@pytest.mark.parametrize("M", [1, 40, 200, 700, 1500])
def test_every_scale_byte_and_code(fmt, M):
    """Scale bytes over the whole range (products that stay in fp32), every pair of codes."""
    N, K = 256, 512
    rng = np.random.default_rng(M)
    a, w = form(M, K, fmt, 3, False), form(N, K, fmt, 4, False)
    if fmt == "mxfp4":
        a, w = (a[0], rng.integers(60, 190, a[1].shape).astype(np.uint8)), (w[0], rng.integers(100, 150, w[1].shape).astype(np.uint8))
    d = sgq.fp4_gemm(*on_gpu(*a), *on_gpu(*w), fmt)
    ok()
    ref.check_product(d, ref.values(*a, fmt), ref.values(*w, fmt), 1.0, torch.bfloat16, f"{fmt} {M}")


@BOTH
@pytest.mark.parametrize("M", [3, 70, 600, 1200])
def test_not_a_number_stays_in_its_row(fmt, M):
    """A group with a NaN scale makes its token's row NaN (or its weight row's column), and nothing else."""
    N, K = 200, 512
    a, w = form(M, K, fmt, 5, True), form(N, K, fmt, 6, True)
    a[1][M // 2, 3] = w[1][77, 1] = 255 if fmt == "mxfp4" else 0x7F
    d = sgq.fp4_gemm(*on_gpu(*a), *on_gpu(*w), fmt)
    ok()
    nan = torch.isnan(d).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2], want[:, 77] = True, True
    assert torch.equal(nan, want)


def test_zero_tokens():
    q, s = sgq.quant_fp4(randn(0, 64), "nvfp4")
    w = sgq.quant_fp4(randn(16, 64), "nvfp4")
    assert q.shape == (0, 32) and sgq.fp4_gemm(q, s, *w, "nvfp4").shape == (0, 16)
    assert sgq.dequant_fp4(q, s, "nvfp4").shape == (0, 64)
    ok()


# ---------------------------------------------------------------- as a program uses them

def block(x, residual, wts, norm, fmt):
    """norm -> gate and up -> silu * up -> down -> residual and next norm, all linears in 4 bits."""
    (gu, gs), (dn, ds) = wts
    q, s = sgq.rms_norm(x, norm, quant=fmt)
    y = sgq.fp4_gemm(q, s, gu, gs, fmt)
    q, s = sgq.quant_fp4(y, fmt, silu_mul=True)
    return sgq.norm_add(sgq.fp4_gemm(q, s, dn, ds, fmt), residual, weight=norm)


def block_parts(M, fmt, seed=0):
    H, I = 512, 768
    wts = [sgq.quant_fp4(randn(2 * I, H, seed=seed + 1, std=0.05), fmt), sgq.quant_fp4(randn(H, I, seed=seed + 2, std=0.05), fmt)]
    return randn(M, H, seed=seed + 3), randn(M, H, seed=seed + 4), wts, randn(H, seed=seed + 5, std=0.1) + 1.0


@BOTH
@pytest.mark.parametrize("M", [1, 50, 700])
def test_block_against_its_steps_in_64_bits(fmt, M):
    """Each step from what the step before it gave, so that no step's error is another's."""
    x, r, wts, n = block_parts(M, fmt)
    h, y = block(x, r, wts, n, fmt)
    ok()
    G = ref.GROUP[fmt]
    of = lambda q, s: ref.values(ref.unpack(q), ref.from_tiles(s, q.shape[0], 2 * q.shape[1] // G), fmt)  # noqa: E731
    q, s = sgq.rms_norm(x, n, quant=fmt)
    ref.check_codes(ref.unpack(q), ref.from_tiles(s, M, 512 // G), ref.norm(ref.f64(x), ref.f64(n), 1e-6, 0.0), fmt, np.float32(1), ref.NORM)
    up = sgq.fp4_gemm(q, s, *wts[0], fmt)
    ref.check_product(up, of(q, s), of(*wts[0]), 1.0, torch.bfloat16)
    q, s = sgq.quant_fp4(up, fmt, silu_mul=True)
    down = sgq.fp4_gemm(q, s, *wts[1], fmt)
    ref.check_product(down, of(q, s), of(*wts[1]), 1.0, torch.bfloat16)
    h2, y2 = sgq.norm_add(down, r, weight=n)
    assert torch.equal(h, h2) and torch.equal(y, y2)


@BOTH
def test_block_in_a_graph_and_eagerly(fmt):
    """A captured block, replayed on new inputs between eager calls, gives the eager bits; so do two graphs in turn."""
    x, r, wts, n = block_parts(300, fmt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            block(x, r, wts, n, fmt)
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                got = block(x, r, wts, n, fmt)
        graphs.append((g, got))
    torch.cuda.synchronize()
    for seed in range(3):
        x.copy_(randn(300, 512, seed=50 + seed))
        for g, _ in graphs:
            g.replay()
        want = block(x, r, wts, n, fmt)
        torch.cuda.synchronize()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    ok()


@BOTH
def test_two_streams_at_once(fmt):
    """Blocks on two streams, with nothing shared but the weights: the bits of each alone."""
    parts = [block_parts(m, fmt, seed=0) for m in (40, 900)]
    want = [block(*p, fmt) for p in parts]
    streams = [torch.cuda.Stream() for _ in parts]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (s, p) in enumerate(zip(streams, parts)):
            with torch.cuda.stream(s):
                got[i].append(block(*p, fmt))
    ok()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for pair in g for a, b in zip(pair, w))


@BOTH
def test_stream_argument(fmt):
    """stream=...: outputs belong to that stream; a raw handle does as well."""
    x, w = randn(200, 256, seed=9), sgq.quant_fp4(randn(64, 256, seed=8), fmt)
    want = sgq.fp4_gemm(*sgq.quant_fp4(x, fmt), *w, fmt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        q = sgq.quant_fp4(x, fmt, stream=stream)
        d = sgq.fp4_gemm(*q, *w, fmt, stream=stream)
        v = sgq.dequant_fp4(*q, fmt, stream=stream)
        s.synchronize()
        assert torch.equal(d, want) and v.shape == x.shape
    ok()


def test_weights_written_by_the_call_before():
    """The product may follow the quantisation of its own weights without a host synchronisation."""
    x = sgq.quant_fp4(randn(64, 2048, seed=1), "nvfp4")
    want = [sgq.fp4_gemm(*x, *sgq.quant_fp4(randn(7168, 2048, seed=s, std=0.02), "nvfp4"), "nvfp4") for s in (2, 3)]
    raw = [randn(7168, 2048, seed=s, std=0.02) for s in (2, 3)]
    wq, ws = sgq.quant_fp4(raw[0], "nvfp4")
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            sgq.quant_fp4(raw[i], "nvfp4", xq=wq, xs=ws)
            assert torch.equal(sgq.fp4_gemm(*x, wq, ws, "nvfp4"), want[i])
    ok()


@BOTH
def test_offsets_past_32_bits(fmt):
    """Every 997 rows of x are the same rows, so those of each output are; 4.4e9 elements of x, 2.2e9 of D."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    R, T, K, N = 997, 612, 7168, 3520
    M = R * T
    base = randn(R, K, seed=1)
    x = base.repeat(T, 1)
    q, s = sgq.quant_fp4(x, fmt)
    del x
    bq, bs = sgq.quant_fp4(base, fmt)
    assert (q.view(T, R, K // 2) == bq).all()
    G = K // ref.GROUP[fmt]
    r, j = torch.arange(M - R, M, device=DEV)[:, None], torch.arange(G, device=DEV)[None]
    assert np.array_equal(s[r // 128, j // 4, r % 32 * 16 + r % 128 // 32 * 4 + j % 4].cpu().numpy(), ref.from_tiles(bs, R, G))
    y, by = sgq.dequant_fp4(q, s, fmt), sgq.dequant_fp4(bq, bs, fmt)
    assert (y.view(T, R, K) == by).all()
    del y
    wq, ws = sgq.quant_fp4(randn(N, K, seed=2, std=0.05), fmt)
    d = sgq.fp4_gemm(q, s, wq, ws, fmt)
    ok()
    assert (d.view(T, R, N) == d[:R]).all()
    ref.check_product(d[-R:], ref.values(ref.unpack(bq), ref.from_tiles(bs, R, G), fmt), ref.values(ref.unpack(wq), ref.from_tiles(ws, N, G), fmt),
                  1.0, torch.bfloat16, fmt)


def test_nothing_is_allocated_by_the_library():
    before = sgq.sgq_allocated_bytes()
    w = sgq.quant_fp4(randn(1536, 7168, seed=1), "mxfp4")
    sgq.fp4_gemm(*sgq.quant_fp4(randn(1, 7168, seed=2), "mxfp4"), *w, "mxfp4")
    ok()
    assert sgq.sgq_allocated_bytes() == before


@pytest.mark.parametrize("M,N,K", [(40, 512, 4096), (300, 2048, 2048), (1100, 4096, 2048)])
def test_wait_that_runs_out(M, N, K):
    """A stage that never comes: the call returns, the status says so once, and the next calls give what they gave before
    (tiles whose K is split over a cluster, pairs with one half and with two)."""
    from fp8_block_scaled_sgq_gb300 import binding
    a, w = on_gpu(*form(M, K, "nvfp4", 1, True)), on_gpu(*form(N, K, "nvfp4", 2, True))
    want = sgq.fp4_gemm(*a, *w, "nvfp4")
    ok()
    d = torch.empty_like(want)
    for _ in range(2):
        sgq.sgq_fp4_gemm(a[0], a[1], None, w[0], w[1], None, d, M, N, K, sgq.SGQ_NVFP4 | binding.SGQ_FP4_TEST_TIMEOUT, sgq.SGQ_BF16)
        assert sgq.sgq_device_status() == binding.SGQ_ERR_TIMEOUT
        assert sgq.sgq_device_status() == 0
        assert torch.equal(sgq.fp4_gemm(*a, *w, "nvfp4"), want)
    ok()


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has to be called once before a graph is captured."""
    code = """
import sys
import torch
sys.path.insert(0, %r)
import fp8_block_scaled_sgq_gb300 as sgq
x, w = torch.randn(96, 512, device="cuda").bfloat16(), torch.randn(1024, 512, device="cuda").bfloat16()
n = torch.ones(512, device="cuda").bfloat16()
def f():
    q = sgq.rms_norm(x, n, quant="nvfp4")
    wq = sgq.quant_fp4(w, "nvfp4")
    return sgq.fp4_gemm(*q, *wq, "nvfp4"), sgq.dequant_fp4(*q, "nvfp4"), sgq.norm_add(x, x, weight=n)[1]
side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
    got = f()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, f()))
print("same")
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
