"""Fused norms on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
import fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])


def ok():
    torch.cuda.synchronize()
    assert sgq.sgq_device_status() == 0


def randn(*shape, seed=0, dtype=torch.bfloat16, std=1.0, mean=0.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(DEV)


def check_rounded(got, want, mag, dtype, what):
    """got: want rounded once, after fp32 arithmetic on terms of magnitude mag."""
    tol = ref.UNIT[dtype] * np.abs(want) + ref.NORM * mag + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = np.abs(ref.f64(got) - want)
    assert np.isfinite(ref.f64(got)).all() and (err <= tol).all(), f"{what}: off by {(err - tol).max()} past the bound"


def check_fp8(codes, scales, y, group, kind, what):
    """FP8 groups of values that are within NORM of y."""
    q = codes.cpu().view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    part = np.abs(y).reshape(y.shape[0], -1, group)
    amax = np.maximum(part.max(axis=-1), 1e-10) / 448
    if kind == "bytes":
        s = 2.0 ** (scales.cpu().numpy().astype(np.float64) - 127)
    else:
        s = ref.f64(scales)
    if kind == "fp32":
        assert (np.abs(s - amax) <= (ref.NORM + 2.0 ** -23) * amax).all(), f"{what}: scales"
    else:
        lo, hi = (2.0 ** np.ceil(np.log2(amax * f)) for f in (1 - 2 * ref.NORM, 1 + 2 * ref.NORM))
        assert ((s >= lo) & (s <= hi)).all(), f"{what}: scales"
    big = np.repeat(s, group, axis=1)
    tol = np.maximum(np.abs(y) * 2.0 ** -4, big * 2.0 ** -10) + 4 * ref.NORM * np.abs(y)     # half a step of E4M3
    assert (np.abs(q * big - y) <= tol).all(), f"{what}: codes"


def run(M, K, dtype, add, post, gate, quant, group=128, ue8m0=False, offset=0.0, eps=1e-6, strided=False, in_place=None, seed=0):
    wide = K + 64 if strided else K
    x, r = randn(M, wide, seed=seed, dtype=dtype)[:, :K], randn(M, wide, seed=seed + 1, dtype=dtype, std=3.0)[:, wide - K:]
    w, p = (randn(K, seed=seed + s, dtype=dtype, std=0.2, mean=1.0 - offset) for s in (2, 3))
    G = {"none": 0, "all": 1, "token": M, "some": next(d for d in (7, 5, 4, 3, 2, 1) if M % d == 0)}[gate]
    g = randn(G, K, seed=seed + 4, dtype=dtype) if G else None
    t = torch.full((1,), 0.0021, device=DEV) if quant == "nvfp4" else None
    kw = dict(eps=eps, offset=offset, quant=quant, tensor_scale=t)
    if quant and quant.startswith("fp8"):
        kw.update(group=group, ue8m0=ue8m0)
    # all rows where they are few, else the first and last of them and some between: rows do not depend on each other
    rows = np.arange(M) if M * K < 2_000_000 else np.unique(np.concatenate([[0, 1, M - 2, M - 1], np.random.default_rng(M).integers(0, M, 40)]))
    at = torch.from_numpy(rows).to(DEV)
    x0, r0, x1, r1 = ref.f64(x[at]), ref.f64(r[at]), x.clone(), r.clone()
    if not add:
        got = sgq.rms_norm(x, w, **kw)
        h, got = x0, got if quant else (got,)
    else:
        out = {None: None, "residual": r, "x": x}[in_place]
        res = sgq.norm_add(x, r, post_weight=p if post else None, gate=g, scale=0.75, residual_scale=1.5, weight=w, h_out=out, **kw)
        assert in_place is None or res[0] is out
        ok()
        u = ref.norm(x0, ref.f64(p), eps, offset) if post else x0
        if G:
            u = u * ref.f64(g)[rows * G // M]
        want = 1.5 * r0 + 0.75 * u
        check_rounded(res[0][at], want, np.abs(1.5 * r0) + np.abs(0.75 * u), dtype, "h")
        assert torch.isfinite(res[0]).all()
        h, got = ref.f64(res[0][at]), res[1:]
        if in_place != "x":
            assert torch.equal(x, x1)
        if in_place != "residual":
            assert torch.equal(r, r1)
    ok()
    y = ref.norm(h, ref.f64(w), eps, offset)
    what = f"{M}x{K} {quant}"
    if quant is None:
        check_rounded(got[0][at], y, np.abs(y), dtype, what)
        assert torch.isfinite(got[0]).all()
    elif quant.startswith("fp8"):
        check_fp8(got[0][at], got[1][at], y, group, "bytes" if quant == "fp8_ue8m0" else "pow2" if ue8m0 else "fp32", what)
    else:
        tiles = ref.from_tiles(got[1], M, got[1].shape[1] * 4)
        ref.check_codes(ref.unpack(got[0][at]), tiles[rows, :K // ref.GROUP[quant]], y, quant,
                        np.float32(0.0021) if t is not None else np.float32(1), ref.NORM, what)
        assert (tiles[:, K // ref.GROUP[quant]:] == 0).all()


def walking(K):
    """Rows that are enough for CTAs that walk over them (more than 10 Mi elements; a warp a row up to 1024 columns)."""
    return 10 * 2 ** 20 // K + 3 if 1024 < K <= 16384 else 700


#: Widths at the kernels' borders (a warp a row up to 1024, a CTA up to 32768), odd ones.
WIDTHS = [8, 24, 1024, 1032, 1536, 1544, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 16384, 16392, 32768]


@TYPES
@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("M", [1, 6, 611, "walking"])
def test_norm_of_every_width(dtype, K, M):
    M = walking(K) if M == "walking" else M
    run(M, K, dtype, False, False, "none", None, offset=1.0)
    run(M, K, dtype, True, True, "some", None)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("add,post,gate", [(False, False, "none"), (True, False, "none"), (True, True, "none"), (True, False, "token"),
                                           (True, True, "all"), (True, True, "some")])
@pytest.mark.parametrize("quant,kw", [(None, {}), ("fp8", dict(group=128)), ("fp8", dict(group=32)), ("fp8", dict(group=32, ue8m0=True)),
                                      ("fp8_ue8m0", dict(group=128)), ("fp8_ue8m0", dict(group=32)), ("mxfp4", {}), ("nvfp4", {})])
def test_every_step_and_form(many, add, post, gate, quant, kw):
    for K in (896, 1536, 4224, 7168):
        run(walking(K) if many else 5, K, torch.bfloat16 if K != 1536 else torch.float16, add, post, gate, quant, **kw)


@pytest.mark.parametrize("quant", [None, "fp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [32, 64, 128, 160, 256, 288, 512, 544, 768, 1024])
@pytest.mark.parametrize("M", [9731, 41002])
def test_many_narrow_rows(quant, K, M):
    """More rows than fit at once: several a warp and step, the last step not whole; in place, too."""
    kw = dict(group=32) if quant == "fp8" else {}
    run(M, K, torch.bfloat16, False, False, "none", quant, **kw)
    run(M, K, torch.bfloat16, True, True, "token" if M < 10000 else "some", quant, in_place="residual", **kw)


@pytest.mark.parametrize("quant", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [32, 96, 1056, 7200, 9248, 32768])
@pytest.mark.parametrize("M", [3, 320, "walking"])
def test_four_bits_of_ragged_rows(quant, K, M):
    run(walking(K) if M == "walking" else M, K, torch.bfloat16, True, False, "none", quant)


@pytest.mark.parametrize("M", [5, 700, "walking"])
@pytest.mark.parametrize("in_place", [None, "residual", "x"])
def test_rows_apart_and_in_place(M, in_place):
    for K in (512, 1544, 7168):
        run(walking(K) if M == "walking" else M, K, torch.bfloat16, True, True, "some", None, strided=True, in_place=in_place)


@pytest.mark.parametrize("M,K", [(3, 256), (400, 2304), (4600, 2304)])
def test_same_codes_as_the_quantisers_on_exact_values(M, K):
    """Rows of +-1 and zeros with weights that are powers of two: with eps 0 the norm is exact where half the row is zero
    (mean 1/4: 1/sqrt is 2), so that it gives what the quantisers give for the same values."""
    sign = (torch.randint(0, 2, (M, K), generator=torch.Generator().manual_seed(1)) * 2 - 1).bfloat16()
    sign[:, ::4], sign[:, 1::4], sign[:, 2::4] = 0, 0, 0
    x, w = sign.to(DEV), (2.0 ** torch.randint(-3, 4, (K,)).float()).bfloat16().to(DEV)
    y = sgq.rms_norm(x, w, eps=0.0)
    assert torch.equal(y, 2 * x * w)
    for quant, other in (("fp8", lambda: sgq.quant_token_group(y, 128, False)), ("fp8_ue8m0", lambda: sgq.quant_token_group_ue8m0(y, 128)),
                         ("mxfp4", lambda: sgq.quant_fp4(y, "mxfp4")), ("nvfp4", lambda: sgq.quant_fp4(y, "nvfp4"))):
        a, b = sgq.rms_norm(x, w, eps=0.0, quant=quant), other()
        G = K // (ref.GROUP.get(quant, 128))
        assert torch.equal(a[0], b[0]), quant
        if quant in ref.GROUP:
            assert np.array_equal(ref.from_tiles(a[1], M, G), ref.from_tiles(b[1], M, G))
        else:
            assert torch.equal(a[1], b[1])
    ok()


@pytest.mark.parametrize("M", [4, 600, 5200])
def test_rows_that_are_not_finite_and_rows_of_zeros(M):
    K = 2048
    x = randn(M, K, seed=3)
    x[0, 5], x[1, 7], x[2] = float("nan"), float("inf"), 0
    w = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    y = sgq.rms_norm(x, w)
    assert torch.isnan(y[0]).all() and torch.isnan(y[1, 7]) and (y[2] == 0).all() and torch.isfinite(y[3:]).all()
    assert (sgq.rms_norm(x[2:3], w, eps=0.0).isnan()).all()        # 0 / 0
    q, s = sgq.rms_norm(x, w, quant="mxfp4")
    v = sgq.dequant_fp4(q, s, "mxfp4")
    assert torch.isnan(v[0]).all() and (v[2] == 0).all() and torch.isfinite(v[3:]).all()
    ok()


@pytest.mark.parametrize("M,K", [(3, 384), (5, 1408), (6900, 1664), (10300, 1536)])
@pytest.mark.parametrize("quant,kw", [("fp8", {}), ("fp8", dict(ue8m0=True)), ("fp8_ue8m0", {})])
def test_fp8_groups_with_weights_that_are_not_finite(M, K, quant, kw):
    """The FP8 quantisers' rule: a group's NaNs leave its scale to its other values, an infinity is one of them."""
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    w = torch.full((K,), 2.0, dtype=torch.bfloat16, device=DEV)
    clean = sgq.rms_norm(x, w, eps=0.0, quant=quant, **kw)
    w[5], w[130], w[256:384] = float("nan"), float("-inf"), float("nan")
    q, s = sgq.rms_norm(x, w, eps=0.0, quant=quant, **kw)
    ok()
    nan = torch.zeros(K, dtype=torch.bool, device=DEV)
    nan[5] = nan[130] = True
    nan[256:384] = True
    assert torch.equal((q & 0x7F) == 0x7F, nan.expand(M, K))                     # NaN, and infinity / infinity
    assert ((q[:, 128:256] & 0x7F)[:, ~nan[128:256]] == 0).all()                 # finite / infinity
    keep = ~nan
    keep[128:256] = False
    assert torch.equal(q[:, keep], clean[0][:, keep])
    assert torch.equal(s[:, 0], clean[1][:, 0]) and torch.equal(s[:, 3:], clean[1][:, 3:])
    assert (s[:, 1] == 255).all() if quant == "fp8_ue8m0" else torch.isposinf(s[:, 1].float()).all()
    zero = sgq.rms_norm(torch.zeros_like(x), w.nan_to_num(1.0, 1.0, 1.0), quant=quant, **kw)[1]
    assert torch.equal(s[:, 2], zero[:, 2])                                      # no number at all: the smallest scale


@pytest.mark.parametrize("M,K", [(3, 384), (6900, 1664), (10300, 1536)])
def test_nvfp4_scales_past_the_reciprocals_range(M, K):
    """Rows of ones with eps 0: y is the weights, exactly; values and tensor scales down to fp32's smallest."""
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    sizes = 2.0 ** torch.linspace(-133, -120, K // 16)
    w = (randn(K, seed=4).float().cpu().view(-1, 16) * sizes[:, None]).flatten().bfloat16()
    w = w + 0.0                     # (no zero has a sign here: w + offset has none)
    w[16:32] = 0
    for t in (2.0 ** -126, 2.0 ** -131, 2.0 ** -149, 2.0 ** 120):
        y = w if t < 1 else (w.double() * 2.0 ** 240).bfloat16()
        q, s = sgq.rms_norm(x, y.to(DEV), eps=0.0, quant="nvfp4", tensor_scale=torch.full((1,), t, device=DEV))
        ok()
        nib, byte = ref.quantise(y.float().numpy()[None], "nvfp4", np.float32(t))
        rows = slice(None) if M < 10 else [0, 1, M // 2, M - 1]
        got = ref.unpack(q[rows])
        assert (got == nib).all(), t
        assert (ref.from_tiles(s, M, K // 16)[rows] == byte).all(), t


def test_outputs_between_guards():
    """Given outputs are written to their borders and not past them."""
    for M, K in ((3, 96), (310, 1120), (9400, 1120)):
        x, r, w = randn(M, K, seed=1), randn(M, K, seed=2), randn(K, seed=3, mean=1.0)
        want = sgq.norm_add(x, r, weight=w, quant="nvfp4")
        hb = torch.full((M * K + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        T = want[2].shape
        qb, sb = (torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV) for n in (M * K // 2, T.numel()))
        got = sgq.norm_add(x, r, weight=w, quant="nvfp4", h_out=hb[32:-32].view(M, K), out=qb[32:-32].view(M, K // 2),
                           out_scales=sb[32:-32].view(T))
        ok()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        G = T[1] * 4
        assert np.array_equal(ref.from_tiles(got[2], M, G), ref.from_tiles(want[2], M, G))
        for b, v in ((hb, 7.0), (qb, 0xA5), (sb, 0xA5)):
            assert (b[:32] == v).all() and (b[-32:] == v).all()


@pytest.mark.parametrize("quant", [None, "fp8", "nvfp4"])
def test_offsets_past_32_bits(quant):
    """Every 997 rows are the same rows, so those of each output are; 4.4e9 elements of x and of h."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    R, T, K = 997, 612, 7168
    base, res, w = randn(R, K, seed=1), randn(R, K, seed=2), randn(K, seed=3, std=0.2, mean=1.0)
    got = sgq.norm_add(base.repeat(T, 1), res.repeat(T, 1), weight=w, quant=quant)
    ok()
    for g in got[:2] if quant == "nvfp4" else got:
        assert (g.view(T, R, -1) == g[:R]).all()
    assert torch.equal(got[0][:R], sgq.norm_add(base, res))
    if quant == "nvfp4":
        G, M = K // 16, R * T
        r, j = torch.arange(M - R, M, device=DEV)[:, None], torch.arange(G, device=DEV)[None]
        last = got[2][r // 128, j // 4, r % 32 * 16 + r % 128 // 32 * 4 + j % 4].cpu().numpy()
        assert np.array_equal(last, ref.from_tiles(got[2], R, G))
    elif quant is None:
        y = ref.norm(ref.f64(got[0][-R:]), ref.f64(w), 1e-6, 0.0)
        check_rounded(got[1][-R:], y, np.abs(y), torch.bfloat16, "y")


def test_feeds_the_fp8_linear():
    """The norm's FP8 groups are what the block-scaled GEMM reads: the same D as from quantising what they stand for."""
    M, N, K = 64, 512, 2048
    x, w, n = randn(M, K, seed=1), randn(N, K, seed=2, std=0.02), randn(K, seed=3, std=0.1, mean=1.0)
    wq, ws = sgq.quant_weight_block(w, 128, 128, True)
    torch.cuda.synchronize()
    q, s = sgq.rms_norm(x, n, quant="fp8", group=128, ue8m0=True)
    d = sgq.fp8_block_gemm(q, s, wq, ws, 128, 128)
    ok()
    a = q.cpu().view(torch.float8_e4m3fn).double().numpy() * np.repeat(ref.f64(s), 128, axis=1)
    b = wq.cpu().view(torch.float8_e4m3fn).double().numpy() * np.repeat(np.repeat(ref.f64(ws), 128, axis=1), 128, axis=0)[:N]
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert (np.abs(ref.f64(d) - want) <= 2.0 ** -8 * np.abs(want) + 1e-4 * mag).all()
