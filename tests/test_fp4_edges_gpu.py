"""4-bit linears and the norms into 4 bits on the GPU, where values or tensor scales are at the ends of fp32."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
import fp4_ref as ref
from test_fp4_gpu import check_quant, ok, on_gpu, one

pytestmark = pytest.mark.gpu
DEV = "cuda"

#: Tensor scales and a group's largest magnitude, of which amax / (6 t) is past fp32's largest value, next to it on both
#: sides, or far below it.
FAR = [(1e-2, 3e38), (1e-10, 1e30), (2.0 ** -61, 2.0 ** 70), (2.0 ** -20, 2.0 ** 120), (2.0 ** -57, 2.0 ** 73.7), (2.0 ** -57, 2.0 ** 73.5),
       (2.0 ** -57, 2.0 ** 20), (2.0 ** -70, 2.0 ** 100)]


def groups(rows, K, top, seed=0):
    """bf16 [rows, K]: groups of 16 with values up to `top`, of both signs; among them groups of small values, of zeros, with a NaN
    and with an infinity."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.rand(rows, K // 16, 16, generator=g, dtype=torch.float64) * 1.9 - 0.95) * top
    x[..., 0] = top * torch.where(torch.rand(rows, K // 16, generator=g) < 0.5, -1.0, 1.0).double()
    x[:, 1] *= 1e-30
    x[:, 2] = 0
    x = x.clamp(-3.3e38, 3.3e38).flatten(1).bfloat16()
    if rows > 2:
        x[1, 5], x[2, K - 1] = float("nan"), -float("inf")
    return x


# ---------------------------------------------------------------- groups far past their tensor scale saturate

@pytest.mark.parametrize("t,top", FAR)
@pytest.mark.parametrize("M,K", [(1, 64), (5, 512), (300, 1056)])
def test_quant_of_groups_far_past_their_tensor_scale(t, top, M, K):
    """s = min(amax / (6 t), 448) and codes of +-6, however large the quotient is: no finite group becomes NaN."""
    x = groups(M, K, top)
    q, s = check_quant(x.to(DEV), "nvfp4", t)
    finite = torch.isfinite(x).view(M, -1, 16).all(-1).numpy()
    byte = ref.from_tiles(s, M, K // 16)
    assert ((byte == 0x7F) == ~finite).all()


@pytest.mark.parametrize("t,top", FAR)
@pytest.mark.parametrize("M,K", [(1, 64), (300, 1056)])
def test_silu_of_groups_far_past_their_tensor_scale(t, top, M, K):
    """silu(32) is 32 within 2^-46, so values are 32 u within 2^-17."""
    u = groups(M, K, top / 40)
    x = torch.cat([torch.full_like(u, 32.0), u], 1).to(DEV)
    q, s = sgq.quant_fp4(x, "nvfp4", tensor_scale=one(t), silu_mul=True)
    ok()
    finite = torch.isfinite(u).view(M, -1, 16).all(-1).numpy()
    nib, byte = ref.unpack(q), ref.from_tiles(s, M, K // 16)
    assert ((byte == 0x7F) == ~finite).all()
    bad = np.repeat(~finite, 16, axis=1)
    assert (nib[bad] == 0).all()
    rows = finite.all(axis=1)
    with np.errstate(over="ignore"):
        ref.check_codes(nib[rows], byte[rows], 32 * ref.f64(u)[rows], "nvfp4", np.float32(t), 2.0 ** -17)


@pytest.mark.parametrize("t,top", FAR)
@pytest.mark.parametrize("M,K", [(3, 384), (41002, 128), (6900, 1664), (10300, 1536)])
def test_norm_of_groups_far_past_their_tensor_scale(t, top, M, K):
    """Rows of ones with eps 0: y is the weights, exactly (a CTA a row, narrow rows, CTAs that walk)."""
    w = groups(1, K, top)[0] + 0.0                  # (w + offset: no zero has a sign)
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    q, s = sgq.rms_norm(x, w.to(DEV), eps=0.0, quant="nvfp4", tensor_scale=one(t))
    ok()
    nib, byte = ref.quantise(w.float().numpy()[None], "nvfp4", np.float32(t))
    rows = slice(None) if M < 10 else [0, 1, M // 2, M - 1]
    assert (ref.from_tiles(s, M, K // 16)[rows] == byte).all()
    assert (ref.unpack(q[rows]) == nib).all()


def test_a_value_that_is_not_finite_is_its_own_groups():
    """Codes, scales and products beside an infinity and a NaN are those of the tensor without them."""
    x, w = groups(1, 512, 3.0).to(DEV).expand(130, 512).contiguous(), sgq.quant_fp4(groups(64, 512, 0.1).nan_to_num(0, 0, 0).to(DEV), "nvfp4")
    bad = x.clone()
    bad[7, 100], bad[9, 300] = float("inf"), float("nan")
    got = []
    for v in (x, bad):
        t = sgq.fp4_tensor_scale(v)
        q, s = sgq.quant_fp4(v, "nvfp4", tensor_scale=t)
        got.append((t, q, ref.from_tiles(s, 130, 32), sgq.fp4_gemm(q, s, *w, "nvfp4", x_scale=t)))
    ok()
    assert torch.equal(got[0][0], got[1][0])
    rows = [r for r in range(130) if r not in (7, 9)]
    assert torch.equal(got[0][1][rows], got[1][1][rows]) and (got[0][2][rows] == got[1][2][rows]).all()
    assert torch.equal(got[0][3][rows], got[1][3][rows]) and torch.isnan(got[1][3][[7, 9]]).all()
    assert (got[1][2] == 0x7F).sum() == 2


# ---------------------------------------------------------------- tensor scales whose product leaves fp32

#: Sizes of each kernel: a tile, tiles whose K is split, pairs with 256 and with 512 tokens.
KERNELS = [(3, 8, 96), (40, 512, 4096), (300, 4096, 512), (1300, 4096, 1568)]


@pytest.mark.parametrize("M,N,K", KERNELS)
@pytest.mark.parametrize("swap", [False, True])
def test_product_whose_tensor_scales_product_is_tiny(M, N, K, swap):
    """1.76 2^-149 is no fp32 number, 2^31 times it is."""
    rng = np.random.default_rng(M)
    a, w = ((rng.choice([5, 6, 7], (r, K)).astype(np.uint8), rng.integers(0x70, 0x7F, (r, K // 16)).astype(np.uint8)) for r in (M, N))
    s, t = (1.375 * 2.0 ** -75, 1.28125 * 2.0 ** -74) if not swap else (1.28125 * 2.0 ** -140, 1.375 * 2.0 ** -9)
    d = sgq.fp4_gemm(*on_gpu(*a), *on_gpu(*w), "nvfp4", x_scale=one(s), w_scale=one(t))
    ok()
    # bf16's smallest normal number is fp32's, and values below it are 2^-134 off at most
    av, wv, alpha = ref.values(*a, "nvfp4"), ref.values(*w, "nvfp4"), float(np.float32(s)) * float(np.float32(t))
    want, mag = av @ wv.T * alpha, np.abs(av) @ np.abs(wv).T * alpha
    assert (np.abs(want) > 2.0 ** -125).mean() > 0.9
    tol = 2.0 ** -8 * np.abs(want) + (K / 16 * 2.0 ** -23 + 2.0 ** -22) * mag + 2.0 ** -133
    assert (np.abs(ref.f64(d) - want) <= tol).all()


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_product_whose_tensor_scales_product_is_huge(M, N, K):
    """The scales' product is past fp32's largest value, the results are not; a token of zeros gives zeros, not 0 * infinity."""
    rng = np.random.default_rng(M)
    a, w = ((rng.integers(0, 16, (r, K)).astype(np.uint8), np.full((r, K // 16), 1, np.uint8)) for r in (M, N))
    a[0][M // 2] = 0
    s, t = 1.375 * 2.0 ** 69, 1.28125 * 2.0 ** 60
    d = sgq.fp4_gemm(*on_gpu(*a), *on_gpu(*w), "nvfp4", x_scale=one(s), w_scale=one(t))
    ok()
    assert (d[M // 2] == 0).all()
    ref.check_product(d, ref.values(*a, "nvfp4"), ref.values(*w, "nvfp4"), float(np.float32(s)) * float(np.float32(t)), torch.bfloat16)


# ---------------------------------------------------------------- codes are those of the division

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_codes_are_the_divisions_for_divisors_of_every_kind(dtype):
    """Every significand of the type in nine binades up to 6, divided by t, whose significands are 1025 of fp32's (a prime step
    apart).  Each group of 16 begins with 6 t, rounded: its scale byte is 1's, and the divisor t itself."""
    n = {torch.bfloat16: 128, torch.float16: 1024}[dtype]
    x = torch.cat([(1 + torch.arange(n, dtype=torch.float64) / n) * 2.0 ** e for e in range(-6, 3)])
    x = x[x <= 6.0]
    x = torch.cat([x, -x])
    rows = -(-x.numel() // 480)
    x = torch.cat([x, x])[:rows * 480].view(-1, 15)
    x = torch.cat([torch.zeros(x.shape[0], 1), x], 1).view(rows, 512).to(dtype)
    for i in range(0, 1 << 23, 8191):
        t = np.float32(1 + i / (1 << 23))
        x[:, ::16] = 6 * float(t)
        q, s = sgq.quant_fp4(x.to(DEV), "nvfp4", tensor_scale=one(float(t)))
        nib, byte = ref.quantise(x.float().numpy(), "nvfp4", t)
        assert (byte == 0x38).all()
        assert np.array_equal(ref.unpack(q), nib) and np.array_equal(ref.from_tiles(s, rows, 32), byte), i
    ok()
