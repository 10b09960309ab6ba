"""The norms around a block of linears, as functions of torch CUDA tensors: the norm before it, and in one pass what
stands between two blocks (norm of the output, gate, scale, residual, next norm), with the result in 16 bits or
quantised for the linear that reads it.

The work is in ``libsgq.so`` (``include/sgq.h``, sgq_norm).  Tensors are bfloat16 or float16, one type for a call, on
the current device.  Wrong shapes, types or strides raise ValueError before anything is launched, and so does a tensor
that requires a gradient while gradients are recorded, or carries a forward-mode tangent: no derivative is recorded here.
"""
from __future__ import annotations

from . import binding, fp4
from .fp4 import _current, _FORMAT, _new, _NUMBER, _scale
from .latent import _contiguous, _device, _dtype, _dual, _fail


def _target(x, M, K, quant, group, ue8m0, tensor_scale, out, out_scales, stream):
    """(the call's `out`, where y goes, where its scales go)."""
    if quant is None:
        if tensor_scale is not None or out_scales is not None or ue8m0:
            _fail("tensor_scale, out_scales and ue8m0 go with quant")
        if out is None:
            return binding.SGQ_OUT_16, _new((M, K), x.dtype, x, stream), None
        _contiguous("out", out, (M, K), x.dtype)
        _dtype(out)
        return binding.SGQ_OUT_16, out, None
    u8 = fp4.torch.uint8
    if not isinstance(quant, str):
        _fail(f"quant: {quant!r} is none of None, 'fp8', 'fp8_ue8m0', 'mxfp4', 'nvfp4'")
    if quant in _FORMAT:
        if ue8m0:
            _fail("ue8m0 goes with quant='fp8'")
        if K % 32:
            _fail(f"{K} columns are not whole groups of 32")
        t = tensor_scale
        if t is not None and (quant != "nvfp4" or t.dtype is not fp4.torch.float32 or t.numel() != 1 or t.requires_grad
                              or _dual()):
            _scale("tensor_scale", t, quant)
        kind = binding.SGQ_OUT_MXFP4 if quant == "mxfp4" else binding.SGQ_OUT_NVFP4
        shape, scales, kept = (M, K // 2), (-(-M // 128), -(-K // _FORMAT[quant][1]), 512), u8
    elif quant == "fp8" or quant == "fp8_ue8m0":
        if tensor_scale is not None:
            _fail("tensor_scale goes with quant='nvfp4'")
        if group not in (32, 128) or K % group:
            _fail(f"{K} columns are not whole groups of {group}, which is 32 or 128")
        if ue8m0 and quant == "fp8_ue8m0":
            _fail("ue8m0 goes with quant='fp8': 'fp8_ue8m0' writes the scales as bytes")
        kind = binding.SGQ_OUT_FP8 | (binding.SGQ_OUT_GROUP_128 if group == 128 else 0)
        kind |= binding.SGQ_OUT_UE8M0 if quant == "fp8_ue8m0" else binding.SGQ_OUT_POW2 if ue8m0 else 0
        shape, scales, kept = (M, K), (M, K // group), u8 if quant == "fp8_ue8m0" else fp4.torch.float32
    else:
        _fail(f"quant: {quant!r} is none of None, 'fp8', 'fp8_ue8m0', 'mxfp4', 'nvfp4'")
    if out is None:
        out = _new(shape, u8, x, stream)
    else:
        _contiguous("out", out, shape, u8)
    if out_scales is None:
        out_scales = _new(scales, kept, x, stream)
    else:
        _contiguous("out_scales", out_scales, scales, kept)
    return kind, out, out_scales


def _rows(name, t, M, K):
    """Whether t is [M, K], each row contiguous."""
    if t.dim() != 2 or t.shape[0] != M or t.shape[1] != K:
        _fail(f"{name}: expected [{M}, {K}], got {tuple(t.shape)}")
    if t.stride(1) != 1 and K > 1:
        _fail(f"{name}: the last dimension is not contiguous")


def _vector(name, t, K):
    _contiguous(name, t, (K,))


def rms_norm(x, weight, eps: float = 1e-6, offset: float = 0.0, quant=None, group: int = 128, ue8m0: bool = False,
             tensor_scale=None, out=None, out_scales=None, stream=None):
    """The norm before a block: y = x / sqrt(mean(x^2) + eps) * (weight + offset) of every row of x [M, K].

    quant None: y, of x's type.  "fp8": (codes [M, K], fp32 scales [M, K/group]) in the form of ``quant_token_group``
    (ue8m0: powers of two); "fp8_ue8m0": scales as bytes; "mxfp4", "nvfp4": (codes, scale tiles) in that of ``quant_fp4``,
    with tensor_scale.  y is not rounded to 16 bits before it is quantised; it is within 2^-18 of its value, and quotients
    are products with the scale's reciprocal where the quantisers divide, so that a code may be the next one where a
    quotient lies by a border.  out, out_scales: outputs to write to.
    """
    torch = fp4.torch or fp4._load()
    device, handle = _current(stream)
    t, kept = tensor_scale, x.dtype
    dt, shape, strides = _NUMBER.get(kept), x.shape, x.stride()
    if (dt is None or len(shape) != 2 or strides[1] != 1 or weight.dtype is not kept or weight.shape != shape[1:]
            or not weight.is_contiguous() or x.get_device() != device or weight.get_device() != device
            or (t is not None and t.get_device() != device) or out is not None or out_scales is not None
            or (torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad)) or _dual()):
        dt = _dtype(x, weight)
        if x.dim() != 2:
            _fail(f"x: expected [M, K], got {tuple(x.shape)}")
        _rows("x", x, *shape)
        _vector("weight", weight, shape[1])
        _device(x, weight, t, out, out_scales)
    M, K = shape
    kind, y, ys = _target(x, M, K, quant, group, ue8m0, t, out, out_scales, stream)
    rc = (binding._lib or binding.load_library()).sgq_norm(
        x.data_ptr(), strides[0] if M > 1 else K, None, None, 0, 0, None, 0, None, 0, weight.data_ptr(), M, K, eps, offset, 1.0,
        1.0, dt, kind, None if t is None else t.data_ptr(), y.data_ptr(), None if ys is None else ys.data_ptr(), handle)
    if rc:
        binding._check(rc, "sgq_norm")
    return y if ys is None else (y, ys)


def norm_add(x, residual, post_weight=None, gate=None, scale: float = 1.0, residual_scale: float = 1.0, weight=None,
             eps: float = 1e-6, offset: float = 0.0, quant=None, group: int = 128, ue8m0: bool = False, tensor_scale=None,
             h_out=None, out=None, out_scales=None, stream=None):
    """What follows a block whose output is x [M, K], in one pass.

    u = x, or its norm with post_weight; h = residual_scale * residual + scale * gate * u, in x's type; with weight, then
    y = the norm of h, as ``rms_norm`` gives it.  gate: [K], or [G, K], each row for M/G consecutive rows of x.  h_out:
    where h goes (it may be residual, or x).  Returns h without weight, else (h, y) or (h, codes, scales).
    """
    torch = fp4.torch or fp4._load()
    device, handle = _current(stream)
    t, p, w, kept, graded = tensor_scale, post_weight, weight, x.dtype, torch.is_grad_enabled()
    dt, shape, strides = _NUMBER.get(kept), x.shape, x.stride()
    if (dt is None or len(shape) != 2 or strides[1] != 1 or residual.dtype is not kept or residual.shape != shape
            or residual.stride(1) != 1 or x.get_device() != device or residual.get_device() != device
            or (graded and (x.requires_grad or residual.requires_grad))
            or (p is not None and (p.dtype is not kept or p.shape != shape[1:] or not p.is_contiguous()
                                   or p.get_device() != device or (graded and p.requires_grad)))
            or (w is not None and (w.dtype is not kept or w.shape != shape[1:] or not w.is_contiguous()
                                   or w.get_device() != device or (graded and w.requires_grad)))
            or (gate is not None and (gate.dtype is not kept or gate.get_device() != device
                                      or (graded and gate.requires_grad)))
            or (t is not None and t.get_device() != device)
            or h_out is not None or out is not None or out_scales is not None or _dual()):
        dt = _dtype(x, residual, p, gate, w, h_out)
        if x.dim() != 2:
            _fail(f"x: expected [M, K], got {tuple(shape)}")
        _rows("x", x, *shape)
        _rows("residual", residual, *shape)
        if p is not None:
            _vector("post_weight", p, shape[1])
        if w is not None:
            _vector("weight", w, shape[1])
        if h_out is not None:
            _rows("h_out", h_out, *shape)
        _device(x, residual, p, gate, w, t, h_out, out, out_scales)
    M, K = shape
    gs = rows = 0
    if gate is not None:
        if gate.dim() == 1:
            gate = gate[None]
        G = gate.shape[0] if gate.dim() == 2 and gate.shape[1] == K else -1
        if G < 0 or (M % G if G else M):
            _fail(f"gate: expected [K] or [G, K] with G dividing {M}, got {tuple(gate.shape)}")
        gs, unit = gate.stride()
        if unit != 1:
            _rows("gate", gate, G, K)
        gs, rows = gs if G > 1 else K, M // G if M else 1
    if h_out is None:
        h_out, ht = _new(shape, kept, x, stream), K
    else:
        ht = h_out.stride(0) if M > 1 else K
    kind, y, ys = binding.SGQ_OUT_NONE, None, None
    if w is not None:
        kind, y, ys = _target(x, M, K, quant, group, ue8m0, t, out, out_scales, stream)
    elif quant is not None or out is not None or out_scales is not None or t is not None or ue8m0:
        _fail("quant, ue8m0, out, out_scales and tensor_scale go with weight")
    rc = (binding._lib or binding.load_library()).sgq_norm(
        x.data_ptr(), strides[0] if M > 1 else K, None if p is None else p.data_ptr(),
        None if gate is None else gate.data_ptr(), gs, rows, residual.data_ptr(), residual.stride(0) if M > 1 else K,
        h_out.data_ptr(), ht, None if w is None else w.data_ptr(), M, K, eps, offset, scale, residual_scale, dt, kind,
        None if t is None else t.data_ptr(), None if y is None else y.data_ptr(), None if ys is None else ys.data_ptr(), handle)
    if rc:
        binding._check(rc, "sgq_norm")
    return h_out if y is None else (h_out, y) if ys is None else (h_out, y, ys)
