"""The norms around a block of linears, as functions of torch CUDA tensors: the norm before it, and in one pass what
stands between two blocks (norm of the output, gate, scale, residual, next norm), with the result in 16 bits or
quantised for the linear that reads it.

The work is in ``libsgq.so`` (``include/sgq.h``, sgq_norm).  Tensors are bfloat16 or float16, one type for a call, on
the current device.  Wrong shapes, types or strides raise ValueError before anything is launched, and so does a tensor
that requires a gradient while gradients are recorded: none is here.
"""
from __future__ import annotations

from . import binding
from .fp4 import _scale, _tiles
from .latent import _contiguous, _device, _dtype, _empty, _fail, _strides


def _target(x, M, K, quant, group, ue8m0, tensor_scale, out, out_scales, stream):
    """(the call's `out`, where y goes, where its scales go)."""
    import torch
    if quant is None:
        if tensor_scale is not None or out_scales is not None or ue8m0:
            _fail("tensor_scale, out_scales and ue8m0 go with quant")
        if out is None:
            return binding.SGQ_OUT_16, _empty((M, K), x, stream), None
        _contiguous("out", out, (M, K), x.dtype)
        return binding.SGQ_OUT_16, out, None
    if quant in ("mxfp4", "nvfp4"):
        if ue8m0:
            _fail("ue8m0 goes with quant='fp8'")
        if K % 32:
            _fail(f"{K} columns are not whole groups of 32")
        _scale("tensor_scale", tensor_scale, quant)
        kind = binding.SGQ_OUT_MXFP4 if quant == "mxfp4" else binding.SGQ_OUT_NVFP4
        shapes, types = ((M, K // 2), _tiles(M, K, quant)), (torch.uint8, torch.uint8)
    elif quant in ("fp8", "fp8_ue8m0"):
        if tensor_scale is not None:
            _fail("tensor_scale goes with quant='nvfp4'")
        if group not in (32, 128) or K % group:
            _fail(f"{K} columns are not whole groups of {group}, which is 32 or 128")
        if ue8m0 and quant == "fp8_ue8m0":
            _fail("ue8m0 goes with quant='fp8': 'fp8_ue8m0' writes the scales as bytes")
        kind = binding.SGQ_OUT_FP8 | (binding.SGQ_OUT_GROUP_128 if group == 128 else 0)
        kind |= binding.SGQ_OUT_UE8M0 if quant == "fp8_ue8m0" else binding.SGQ_OUT_POW2 if ue8m0 else 0
        shapes = (M, K), (M, K // group)
        types = torch.uint8, torch.uint8 if quant == "fp8_ue8m0" else torch.float32
    else:
        _fail(f"quant: {quant!r} is none of None, 'fp8', 'fp8_ue8m0', 'mxfp4', 'nvfp4'")
    if out is None:
        out = _empty(shapes[0], x, stream, types[0])
    else:
        _contiguous("out", out, shapes[0], types[0])
    if out_scales is None:
        out_scales = _empty(shapes[1], x, stream, types[1])
    else:
        _contiguous("out_scales", out_scales, shapes[1], types[1])
    return kind, out, out_scales


def _rows(name, t, M, K):
    """The row stride of a [M, K] tensor."""
    if t.dim() != 2 or t.shape[0] != M or t.shape[1] != K:
        _fail(f"{name}: expected [{M}, {K}], got {tuple(t.shape)}")
    s, = _strides(name, t, 2)
    return s if M > 1 else K


def _grads(t):
    import torch
    if t is not None and t.requires_grad and torch.is_grad_enabled():
        _fail("tensor_scale requires a gradient, and none is recorded here")


def rms_norm(x, weight, eps: float = 1e-6, offset: float = 0.0, quant=None, group: int = 128, ue8m0: bool = False,
             tensor_scale=None, out=None, out_scales=None, stream=None):
    """The norm before a block: y = x / sqrt(mean(x^2) + eps) * (weight + offset) of every row of x [M, K].

    quant None: y, of x's type.  "fp8": (codes [M, K], fp32 scales [M, K/group]) as ``quant_token_group`` gives them
    (ue8m0: powers of two); "fp8_ue8m0": scales as bytes; "mxfp4", "nvfp4": (codes, scale tiles) as ``quant_fp4`` gives
    them, with tensor_scale.  y is not rounded to 16 bits before it is quantised.  out, out_scales: outputs to write to.
    """
    dt = _dtype(x, weight)
    if x.dim() != 2:
        _fail(f"x: expected [M, K], got {tuple(x.shape)}")
    M, K = x.shape
    xt = _rows("x", x, M, K)
    _contiguous("weight", weight, (K,))
    _grads(tensor_scale)
    _device(x, weight, tensor_scale, out, out_scales)
    kind, y, ys = _target(x, M, K, quant, group, ue8m0, tensor_scale, out, out_scales, stream)
    binding.sgq_norm(x, xt, None, None, 0, 0, None, 0, None, 0, weight, M, K, eps, offset, 1.0, 1.0, dt, kind, tensor_scale,
                     y, ys, stream)
    return y if ys is None else (y, ys)


def norm_add(x, residual, post_weight=None, gate=None, scale: float = 1.0, residual_scale: float = 1.0, weight=None,
             eps: float = 1e-6, offset: float = 0.0, quant=None, group: int = 128, ue8m0: bool = False, tensor_scale=None,
             h_out=None, out=None, out_scales=None, stream=None):
    """What follows a block whose output is x [M, K], in one pass.

    u = x, or its norm with post_weight; h = residual_scale * residual + scale * gate * u, in x's type; with weight, then
    y = the norm of h, as ``rms_norm`` gives it.  gate: [K], or [G, K], each row for M/G consecutive rows of x.  h_out:
    where h goes (it may be residual, or x).  Returns h without weight, else (h, y) or (h, codes, scales).
    """
    dt = _dtype(x, residual, post_weight, gate, weight, h_out)
    if x.dim() != 2:
        _fail(f"x: expected [M, K], got {tuple(x.shape)}")
    M, K = x.shape
    xt, rt = _rows("x", x, M, K), _rows("residual", residual, M, K)
    if post_weight is not None:
        _contiguous("post_weight", post_weight, (K,))
    gs = rows = 0
    if gate is not None:
        if gate.dim() == 1:
            gate = gate[None]
        G = gate.shape[0]
        if gate.dim() != 2 or gate.shape[1] != K or (M % G if G else M):
            _fail(f"gate: expected [K] or [G, K] with G dividing {M}, got {tuple(gate.shape)}")
        (gs,), rows = _strides("gate", gate, 2), M // G if M else 1
        gs = gs if G > 1 else K
    _grads(tensor_scale)
    _device(x, residual, post_weight, gate, weight, tensor_scale, h_out, out, out_scales)
    if h_out is None:
        h_out, ht = _empty((M, K), x, stream), K
    else:
        ht = _rows("h_out", h_out, M, K)
    kind, y, ys = binding.SGQ_OUT_NONE, None, None
    if weight is not None:
        _contiguous("weight", weight, (K,))
        kind, y, ys = _target(x, M, K, quant, group, ue8m0, tensor_scale, out, out_scales, stream)
    elif quant is not None or out is not None or out_scales is not None or tensor_scale is not None:
        _fail("quant, out, out_scales and tensor_scale go with weight")
    binding.sgq_norm(x, xt, post_weight, gate, gs, rows, residual, rt, h_out, ht, weight, M, K, eps, offset, scale,
                     residual_scale, dt, kind, tensor_scale, y, ys, stream)
    return h_out if y is None else (h_out, y) if ys is None else (h_out, y, ys)
