"""4-bit linears and norms without a GPU: tensor scales of unusual tensors, and calls that have to be refused."""
import torch

import fp8_block_scaled_sgq_gb300 as sgq
from test_fp4 import bf, launches, refused  # noqa: F401  (launches: a fixture)


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
