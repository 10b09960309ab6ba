"""Fused norms of wide rows into every quantised form, and what a call repeats, against 64 bits."""
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
from test_norms_gpu import ok, randn, run, walking

pytestmark = pytest.mark.gpu
DEV = "cuda"

#: Past 8192 elements, at the borders of the kernels' widths (8192, 9216, 12288, 16384), where a thread's last column is one for
#: all and where it is not.
WIDE = [8320, 9216, 12288, 12416, 16384]
FORMS = [("fp8", dict(group=128)), ("fp8", dict(group=32, ue8m0=True)), ("fp8_ue8m0", dict(group=32)), ("mxfp4", {}), ("nvfp4", {})]


@pytest.mark.parametrize("quant,kw", FORMS)
@pytest.mark.parametrize("K", WIDE)
@pytest.mark.parametrize("add", [False, True])
def test_many_wide_rows(add, K, quant, kw):
    run(walking(K), K, torch.bfloat16, add, add, "some" if add else "none", quant, **kw)


@pytest.mark.parametrize("quant,kw", FORMS)
@pytest.mark.parametrize("K", [8320, 16384, 16512, 32768])
@pytest.mark.parametrize("M", [2, 160])
def test_few_wide_rows(M, K, quant, kw):
    run(M, K, torch.bfloat16, False, False, "none", quant, **kw)
    run(M, K, torch.float16, True, M > 2, "token", quant, **kw)


@pytest.mark.parametrize("K,quant,kw", [(K, *f) for K in (544, 640, 1024) for f in FORMS if K % f[1].get("group", 32) == 0])
def test_many_rows_of_513_to_1024(K, quant, kw):
    """Enough rows for CTAs that walk over them."""
    M = 10 * 2 ** 20 // K + 3
    run(M, K, torch.bfloat16, False, False, "none", quant, **kw)
    run(M, K, torch.bfloat16, True, True, "token", quant, **kw)


@pytest.mark.parametrize("M,K", [(1, 7168), (4096, 7168), (8191, 1536), (41002, 128), (700, 32768)])
@pytest.mark.parametrize("quant", [None, "fp8", "nvfp4"])
def test_a_call_repeats_itself(M, K, quant):
    """The same bits from every call: sums are taken in one order."""
    x, r, w = randn(M, K, seed=1), randn(M, K, seed=2, std=3.0), randn(K, seed=3, std=0.1, mean=1.0)
    p, g = randn(K, seed=4, std=0.1, mean=1.0), randn(K, seed=5)
    t = torch.full((1,), 0.0021, device=DEV) if quant == "nvfp4" else None
    rows = torch.arange(M, device=DEV)[:, None]
    groups = torch.arange(K // 16, device=DEV)[None]
    want = None
    for _ in range(20):
        got = list(sgq.norm_add(x, r, post_weight=p, gate=g, scale=0.5, residual_scale=1.25, weight=w, quant=quant, tensor_scale=t))
        if quant == "nvfp4":        # (rows past M of the last tile are nobody's)
            got[2] = got[2][rows // 128, groups // 4, rows % 32 * 16 + rows % 128 // 32 * 4 + groups % 4]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ok()
