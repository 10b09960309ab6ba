"""Linears in 4 bits, as functions of torch CUDA tensors: quantisation to E2M1 codes with microscales, its way back,
and the product.

The work is in ``libsgq.so`` (``include/sgq.h``, "4-bit linears"); these helpers check shapes, types and strides and
allocate what they return on the stream of the call.  Formats: "mxfp4" (32 values a scale, a power of two) and "nvfp4"
(16 values a scale, E4M3, and one fp32 scale a tensor).  A tensor of M rows and K columns in that form is two uint8
tensors: codes [M, K/2] and scale tiles [ceil(M/128), T, 512], T = ceil(K/128) ("mxfp4") or ceil(K/64) ("nvfp4").
Wrong shapes, types or strides raise ValueError before anything is launched, and so does a tensor that requires a
gradient while gradients are recorded, or carries a forward-mode tangent: no derivative is recorded here.
"""
from __future__ import annotations

from . import binding
from .latent import _contiguous, _device, _dtype, _dual, _empty, _fail, _no_tangent

torch = None        # imported with the first call: the package itself does without it
_NUMBER = {}        # the C interface's numbers of the element types
_FORMAT = {"mxfp4": (binding.SGQ_MXFP4, 128), "nvfp4": (binding.SGQ_NVFP4, 64)}    # and values of a row in a tile of scales


def _load():
    global torch
    import torch as t
    _NUMBER.update({t.bfloat16: binding.SGQ_BF16, t.float16: binding.SGQ_FP16})
    torch = t
    return t


# The smallest calls take less time on the GPU than their checks do on the host.  So each helper asks everything at
# once, in plain comparisons, and a helper's _why_not finds out what was wrong only when something was.

def _format(fmt):
    try:
        return _FORMAT[fmt]
    except (KeyError, TypeError):
        _fail(f"format {fmt!r} is neither 'mxfp4' nor 'nvfp4'")


def _current(stream):
    """(the current device, the call's stream as a handle)."""
    try:   # (names of this torch that are not public: 0.9 -> 0.2 us)
        device = torch._C._cuda_getDevice()
        if stream is None:
            return device, torch._C._cuda_getCurrentRawStream(device)
    except AttributeError:
        device = torch.cuda.current_device()
    return device, binding._stream(stream)


def _new(shape, dtype, x, stream):
    """A new tensor on x's device that belongs to the call's stream."""
    return torch.empty(shape, dtype=dtype, device=x.device) if stream is None else _empty(shape, x, stream, dtype)


def _scale(name: str, t, fmt):
    """Whether t is a tensor scale: one fp32 value on the device, of the two-level format only."""
    if t is not None:
        if fmt != "nvfp4":
            _fail(f"{name}: 'mxfp4' has no tensor scale")
        if t.dtype != torch.float32 or t.numel() != 1:
            _fail(f"{name}: expected one float32 value, got {tuple(t.shape)} of {t.dtype}")
        if t.requires_grad and torch.is_grad_enabled():
            _fail(f"{name} requires a gradient, and none is recorded here")
        if _dual():
            _no_tangent(t)


def _packed(name: str, q, s, fmt: str):
    """Whether q and s are a tensor in the 4-bit form."""
    if q.dim() != 2 or q.dtype != torch.uint8 or not q.is_contiguous():
        _fail(f"{name}: expected contiguous uint8 codes [rows, K/2], got {tuple(q.shape)} of {q.dtype}")
    M, K = q.shape[0], 2 * q.shape[1]
    _contiguous(f"{name}'s scale tiles", s, (-(-M // 128), -(-K // _FORMAT[fmt][1]), 512), torch.uint8)


def fp4_tensor_scale(x):
    """fp32 [1]: the "nvfp4" tensor scale of x, max|x| / (6 * 448) over its finite values (1 where these are only zeros
    or none): infinities and NaN are for their own groups alone.
    """
    if torch is None:
        _load()
    if x.numel() == 0:
        return torch.ones(1, dtype=torch.float32, device=x.device)
    t = (x.detach().nan_to_num(0.0, 0.0, 0.0).abs().amax().float() / (6.0 * 448.0)).reshape(1)
    return torch.where(t > 0, t.clamp_min(torch.finfo(torch.float32).tiny), torch.ones_like(t))


def fp4_scales_to_tiles(s):
    """Scale bytes uint8 [rows, groups] in rows -> the tiles that the product reads (once, when weights are loaded)."""
    if torch is None:
        _load()
    if s.dim() != 2 or s.dtype != torch.uint8:
        _fail(f"expected uint8 [rows, groups], got {tuple(s.shape)} of {s.dtype}")
    rows, groups = s.shape
    full = torch.zeros(-(-rows // 128) * 128, -(-groups // 4) * 4, dtype=torch.uint8, device=s.device)
    full[:rows, :groups] = s
    tiles = full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return tiles.reshape(full.shape[0] // 128, full.shape[1] // 4, 512)


def fp4_scales_from_tiles(tiles, rows: int, groups: int):
    """The way back: uint8 [rows, groups]."""
    _contiguous("scale tiles", tiles, (-(-rows // 128), -(-groups // 4), 512))
    t = tiles.view(tiles.shape[0], tiles.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(tiles.shape[0] * 128, tiles.shape[1] * 4)[:rows, :groups].contiguous()


def quant_fp4(x, fmt: str, tensor_scale=None, silu_mul: bool = False, xq=None, xs=None, stream=None):
    """x [M, K] (bf16 or fp16, rows any 16-byte multiple apart) -> (codes uint8 [M, K/2], scale tiles uint8).

    silu_mul: x is [M, 2K], rows of [gate | up], and silu(gate) * up is quantised.  tensor_scale: fp32 [1] on the
    device ("nvfp4"; None: 1).  xq, xs: outputs to write to.

    Codes of x are those of fp32 divisions, bit for bit.  silu(gate) * up is within 2^-17 of its value (approximate
    exponential and reciprocal, unlike ``quant_token_group_v2``'s), and its quotients are products with the scale's
    reciprocal, so that a code may be the next one where a quotient lies by a border.
    """
    if torch is None:
        _load()
    f, tile = _format(fmt)
    t, u8, dt = tensor_scale, torch.uint8, _NUMBER.get(x.dtype)
    device, handle = _current(stream)
    shape, strides = x.shape, x.stride()
    if len(shape) != 2 or dt is None or x.get_device() != device:
        _why_not_quant(x, silu_mul, t, fmt, xq, xs)
    M, W = shape
    K = W // 2 if silu_mul else W
    if (strides[1] != 1 or K % 32 or not K or (silu_mul and W % 2) or (x.requires_grad and torch.is_grad_enabled())
            or (t is not None and (t.get_device() != device or fmt != "nvfp4" or t.dtype is not torch.float32
                                   or t.numel() != 1 or t.requires_grad)) or xq is not None or xs is not None or _dual()):
        _why_not_quant(x, silu_mul, t, fmt, xq, xs)
    if xq is None:
        xq = _new((M, K // 2), u8, x, stream)
    if xs is None:
        xs = _new((-(-M // 128), -(-K // tile), 512), u8, x, stream)
    rc = (binding._lib or binding.load_library()).sgq_quant_fp4(
        x.data_ptr(), M, K, strides[0] if M > 1 else W, f, t if t is None else t.data_ptr(), 1 if silu_mul else 0, dt,
        xq.data_ptr(), xs.data_ptr(), handle)
    if rc:
        binding._check(rc, "sgq_quant_fp4")
    return xq, xs


def _why_not_quant(x, silu_mul, t, fmt, xq, xs):
    _dtype(x)
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        _fail(f"x: expected rows of contiguous values, got {tuple(x.shape)} with strides {x.stride()}")
    M, K = x.shape
    if silu_mul:
        if K % 2:
            _fail("x: rows of [gate | up] have an even length")
        K //= 2
    if K % 32 or K == 0:
        _fail(f"{K} columns are not whole groups of 32")
    _scale("tensor_scale", t, fmt)
    _device(x, t, xq, xs)
    if xq is not None:
        _contiguous("xq", xq, (M, K // 2), torch.uint8)
    if xs is not None:
        _contiguous("xs", xs, (-(-M // 128), -(-K // _FORMAT[fmt][1]), 512), torch.uint8)


def dequant_fp4(xq, xs, fmt: str, tensor_scale=None, dtype=None, out=None, stream=None):
    """The values [M, K] that codes and scale tiles stand for, formed in fp32, in bfloat16 (or dtype, or out's type)."""
    if torch is None:
        _load()
    f, tile = _format(fmt)
    t, u8, shape = tensor_scale, torch.uint8, xq.shape
    device, handle = _current(stream)
    dtype = dtype or (torch.bfloat16 if out is None else out.dtype)
    dt = _NUMBER.get(dtype)
    if (len(shape) != 2 or dt is None or xq.dtype is not u8 or xs.dtype is not u8 or not xq.is_contiguous()
            or not xs.is_contiguous() or xs.shape != (-(-shape[0] // 128), -(-2 * shape[1] // tile), 512)
            or xq.get_device() != device or xs.get_device() != device or out is not None
            or (t is not None and (t.get_device() != device or fmt != "nvfp4" or t.dtype is not torch.float32
                                   or t.numel() != 1 or t.requires_grad or _dual()))):
        _packed("xq", xq, xs, fmt)
        _scale("tensor_scale", t, fmt)
        _device(xq, xs, t, out)
        _out(out, dtype, (shape[0], 2 * shape[1]))
    M, K = shape[0], 2 * shape[1]
    if out is None:
        out = _new((M, K), dtype, xq, stream)
    rc = (binding._lib or binding.load_library()).sgq_dequant_fp4(
        xq.data_ptr(), xs.data_ptr(), M, K, f, t if t is None else t.data_ptr(), dt, out.data_ptr(), handle)
    if rc:
        binding._check(rc, "sgq_dequant_fp4")
    return out


def _out(out, dtype, shape):
    if _NUMBER.get(dtype) is None:
        _fail(f"element type {dtype} is neither bfloat16 nor float16")
    if out is not None:
        _contiguous("out", out, shape, dtype)
        _dtype(out)


def fp4_gemm(xq, xs, wq, ws, fmt: str, x_scale=None, w_scale=None, dtype=None, out=None, stream=None):
    """x w^T of two tensors in the 4-bit form: [M, N] in bfloat16 (or dtype, or out's type), fp32 accumulation.

    x_scale, w_scale: the tensors' fp32 scales ("nvfp4"; None: 1).
    """
    if torch is None:
        _load()
    f, tile = _format(fmt)
    a, w, u8, f32, xshape, wshape = x_scale, w_scale, torch.uint8, torch.float32, xq.shape, wq.shape
    device, handle = _current(stream)
    dtype = dtype or (torch.bfloat16 if out is None else out.dtype)
    dt = _NUMBER.get(dtype)
    if (len(xshape) != 2 or len(wshape) != 2 or xshape[1] != wshape[1] or dt is None or xq.dtype is not u8
            or xs.dtype is not u8 or wq.dtype is not u8 or ws.dtype is not u8 or not xq.is_contiguous()
            or not xs.is_contiguous() or not wq.is_contiguous() or not ws.is_contiguous()
            or xs.shape != (-(-xshape[0] // 128), -(-2 * xshape[1] // tile), 512)
            or ws.shape != (-(-wshape[0] // 128), -(-2 * wshape[1] // tile), 512)
            or xq.get_device() != device or xs.get_device() != device or wq.get_device() != device
            or ws.get_device() != device or out is not None
            or (a is not None and (a.get_device() != device or fmt != "nvfp4" or a.dtype is not f32 or a.numel() != 1
                                   or a.requires_grad))
            or (w is not None and (w.get_device() != device or fmt != "nvfp4" or w.dtype is not f32 or w.numel() != 1
                                   or w.requires_grad)) or _dual()):
        _packed("xq", xq, xs, fmt)
        _packed("wq", wq, ws, fmt)
        if xshape[1] != wshape[1]:
            _fail(f"xq has {2 * xshape[1]} columns, wq {2 * wshape[1]}")
        _scale("x_scale", a, fmt)
        _scale("w_scale", w, fmt)
        _device(xq, xs, wq, ws, a, w, out)
        _out(out, dtype, (xshape[0], wshape[0]))
    M, N = xshape[0], wshape[0]
    if out is None:
        out = _new((M, N), dtype, xq, stream)
    rc = (binding._lib or binding.load_library()).sgq_fp4_gemm(
        xq.data_ptr(), xs.data_ptr(), a if a is None else a.data_ptr(), wq.data_ptr(), ws.data_ptr(),
        w if w is None else w.data_ptr(), out.data_ptr(), M, N, 2 * xshape[1], f, dt, handle)
    if rc:
        binding._check(rc, "sgq_fp4_gemm")
    return out
