"""4-bit linears and norms without a GPU: tensor scales of unusual tensors, and calls that have to be refused."""
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
from test_fp4 import bf, launches, refused, u8  # noqa: F401  (launches: a fixture)


def test_tensor_scale_is_of_the_finite_values():
    """An infinity or a NaN makes its own group NaN: the tensor's scale stays positive and finite, the one of the other values."""
    x = torch.tensor([[1.0, -13.44], [0.0, 2.0]]).bfloat16()
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        clean = sgq.fp4_tensor_scale(x.to(dtype))
        for bad in (float("inf"), -float("inf"), float("nan")):
            y = torch.cat([x.to(dtype), torch.full((1, 2), bad, dtype=dtype)])
            assert torch.equal(sgq.fp4_tensor_scale(y), clean)
            assert sgq.fp4_tensor_scale(y[2:]).item() == 1.0


def test_tensor_scale_of_nothing():
    """As for zeros: no tokens are no error anywhere else."""
    for shape in ((0,), (0, 64)):
        t = sgq.fp4_tensor_scale(torch.zeros(shape, dtype=torch.bfloat16))
        assert t.shape == (1,) and t.dtype == torch.float32 and t.item() == 1.0


def test_forms_that_no_dictionary_takes(launches):  # noqa: F811
    x, w = bf(4, 128), bf(128)
    for quant in (["nvfp4"], {"nvfp4"}, {}):
        refused(sgq.rms_norm, x, w, quant=quant)
        refused(sgq.norm_add, x, x, weight=w, quant=quant)
    assert not launches


def test_powers_of_two_go_with_a_form(launches):  # noqa: F811
    """As in rms_norm, an argument that nothing would heed is refused."""
    x = bf(4, 128)
    refused(sgq.norm_add, x, x, ue8m0=True)
    assert not launches


def test_tensors_with_a_tangent_are_refused(launches):  # noqa: F811
    """Forward-mode derivatives are not recorded either, and would be lost without a word."""
    import torch.autograd.forward_ad as ad
    x, w, t, q, s = bf(4, 128), bf(128), torch.ones(1), u8(4, 64), u8(1, 2, 512)
    with ad.dual_level():
        dual = lambda v: ad.make_dual(v, torch.ones_like(v))  # noqa: E731
        dx, dw, dt = dual(x), dual(w), dual(t)
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                refused(sgq.quant_fp4, dx, "nvfp4")
                refused(sgq.quant_fp4, x, "nvfp4", tensor_scale=dt)
                refused(sgq.dequant_fp4, q, s, "nvfp4", tensor_scale=dt)
                refused(sgq.fp4_gemm, q, s, q, s, "nvfp4", x_scale=dt)
                refused(sgq.fp4_gemm, q, s, q, s, "nvfp4", w_scale=dt)
                refused(sgq.rms_norm, dx, w)
                refused(sgq.rms_norm, x, dw)
                refused(sgq.rms_norm, x, w, quant="nvfp4", tensor_scale=dt)
                for k in (dict(x=dx), dict(residual=dx), dict(post_weight=dw), dict(weight=dw), dict(gate=dw),
                          dict(weight=w, quant="nvfp4", tensor_scale=dt)):
                    refused(sgq.norm_add, **{**dict(x=x, residual=x), **k})
        assert not launches
        # others are not in the way of a level
        sgq.rms_norm(x, w)
        sgq.norm_add(x, x, weight=w, gate=w, quant="nvfp4", tensor_scale=t)
        sgq.quant_fp4(x, "nvfp4", tensor_scale=t)
        sgq.fp4_gemm(q, s, u8(8, 64), s, "nvfp4", x_scale=t)
        sgq.dequant_fp4(q, s, "nvfp4", tensor_scale=t)
        assert len(launches) == 5


def test_latent_helpers_refuse_a_tangent():
    """The latent helpers' check is the same one."""
    import torch.autograd.forward_ad as ad
    from fp8_block_scaled_sgq_gb300.latent import _dtype
    with ad.dual_level():
        dx = ad.make_dual(bf(4, 2, 64), torch.ones(4, 2, 64).bfloat16())
        for args in ((dx,), (bf(2), dx)):
            with pytest.raises(ValueError):
                _dtype(*args)
        _dtype(bf(2), bf(2))
