"""Linears in 4 bits, as functions of torch CUDA tensors: quantisation to E2M1 codes with microscales, its way back,
and the product.

The work is in ``libsgq.so`` (``include/sgq.h``, "4-bit linears"); these helpers check shapes, types and strides and
allocate what they return on the stream of the call.  Formats: "mxfp4" (32 values a scale, a power of two) and "nvfp4"
(16 values a scale, E4M3, and one fp32 scale a tensor).  A tensor of M rows and K columns in that form is two uint8
tensors: codes [M, K/2] and scale tiles [ceil(M/128), T, 512], T = ceil(K/128) ("mxfp4") or ceil(K/64) ("nvfp4").
Wrong shapes, types or strides raise ValueError before anything is launched, and so does a tensor that requires a
gradient while gradients are recorded: none is here.
"""
from __future__ import annotations

from . import binding
from .latent import _contiguous, _device, _dtype, _empty, _fail

_FORMAT = {"mxfp4": binding.SGQ_MXFP4, "nvfp4": binding.SGQ_NVFP4}
_TILE_K = {"mxfp4": 128, "nvfp4": 64}     # values of a row in a tile of scales


def _format(fmt) -> int:
    try:
        return _FORMAT[fmt]
    except (KeyError, TypeError):
        _fail(f"format {fmt!r} is neither 'mxfp4' nor 'nvfp4'")


def _tiles(M: int, K: int, fmt: str):
    return -(-M // 128), -(-K // _TILE_K[fmt]), 512


def _scale(name: str, t, fmt: str):
    """A tensor scale: one fp32 value on the device, of the two-level format only."""
    import torch
    if t is not None:
        if fmt != "nvfp4":
            _fail(f"{name}: 'mxfp4' has no tensor scale")
        if t.dtype != torch.float32 or t.numel() != 1:
            _fail(f"{name}: expected one float32 value, got {tuple(t.shape)} of {t.dtype}")
        if t.requires_grad and torch.is_grad_enabled():
            _fail(f"{name} requires a gradient, and none is recorded here")


def _packed(name: str, q, s, fmt: str):
    """(M, K) of a tensor in the 4-bit form."""
    import torch
    if q.dim() != 2 or q.dtype != torch.uint8 or not q.is_contiguous():
        _fail(f"{name}: expected contiguous uint8 codes [rows, K/2], got {tuple(q.shape)} of {q.dtype}")
    M, K = q.shape[0], 2 * q.shape[1]
    _contiguous(f"{name}'s scale tiles", s, _tiles(M, K, fmt), torch.uint8)
    return M, K


def fp4_tensor_scale(x):
    """fp32 [1]: the "nvfp4" tensor scale of x, max|x| / (6 * 448) (1 where x holds only zeros)."""
    import torch
    t = (x.detach().abs().amax().float() / (6.0 * 448.0)).reshape(1)
    return torch.where(t > 0, t.clamp_min(torch.finfo(torch.float32).tiny), torch.ones_like(t))


def fp4_scales_to_tiles(s):
    """Scale bytes uint8 [rows, groups] in rows -> the tiles that the product reads (once, when weights are loaded)."""
    import torch
    if s.dim() != 2 or s.dtype != torch.uint8:
        _fail(f"expected uint8 [rows, groups], got {tuple(s.shape)} of {s.dtype}")
    rows, groups = s.shape
    full = torch.zeros(-(-rows // 128) * 128, -(-groups // 4) * 4, dtype=torch.uint8, device=s.device)
    full[:rows, :groups] = s
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, full.shape[1] // 4, 512)


def fp4_scales_from_tiles(tiles, rows: int, groups: int):
    """The way back: uint8 [rows, groups]."""
    _contiguous("scale tiles", tiles, (-(-rows // 128), -(-groups // 4), 512))
    t = tiles.view(tiles.shape[0], tiles.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(tiles.shape[0] * 128, tiles.shape[1] * 4)[:rows, :groups].contiguous()


def quant_fp4(x, fmt: str, tensor_scale=None, silu_mul: bool = False, xq=None, xs=None, stream=None):
    """x [M, K] (bf16 or fp16, rows any 16-byte multiple apart) -> (codes uint8 [M, K/2], scale tiles uint8).

    silu_mul: x is [M, 2K], rows of [gate | up], and silu(gate) * up is quantised.  tensor_scale: fp32 [1] on the
    device ("nvfp4"; None: 1).  xq, xs: outputs to write to.
    """
    import torch
    f, dt = _format(fmt), _dtype(x)
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        _fail(f"x: expected rows of contiguous values, got {tuple(x.shape)} with strides {x.stride()}")
    M, K = x.shape
    if silu_mul:
        if K % 2:
            _fail("x: rows of [gate | up] have an even length")
        K //= 2
    if K % 32 or K == 0:
        _fail(f"{K} columns are not whole groups of 32")
    _scale("tensor_scale", tensor_scale, fmt)
    _device(x, tensor_scale, xq, xs)
    if xq is None:
        xq = _empty((M, K // 2), x, stream, torch.uint8)
    else:
        _contiguous("xq", xq, (M, K // 2), torch.uint8)
    if xs is None:
        xs = _empty(_tiles(M, K, fmt), x, stream, torch.uint8)
    else:
        _contiguous("xs", xs, _tiles(M, K, fmt), torch.uint8)
    binding.sgq_quant_fp4(x, M, K, x.stride(0) if M > 1 else x.shape[1], f, tensor_scale, silu_mul, dt, xq, xs, stream)
    return xq, xs


def dequant_fp4(xq, xs, fmt: str, tensor_scale=None, dtype=None, out=None, stream=None):
    """The values [M, K] that codes and scale tiles stand for, in bfloat16 (or dtype, or out's type)."""
    import torch
    f = _format(fmt)
    M, K = _packed("xq", xq, xs, fmt)
    _scale("tensor_scale", tensor_scale, fmt)
    _device(xq, xs, tensor_scale, out)
    if out is None:
        out = _empty((M, K), xq, stream, dtype or torch.bfloat16)
    else:
        _contiguous("out", out, (M, K), dtype)
    binding.sgq_dequant_fp4(xq, xs, M, K, f, tensor_scale, _dtype(out), out, stream)
    return out


def fp4_gemm(xq, xs, wq, ws, fmt: str, x_scale=None, w_scale=None, dtype=None, out=None, stream=None):
    """x w^T of two tensors in the 4-bit form: [M, N] in bfloat16 (or dtype, or out's type), fp32 accumulation.

    x_scale, w_scale: the tensors' fp32 scales ("nvfp4"; None: 1).
    """
    import torch
    f = _format(fmt)
    M, K = _packed("xq", xq, xs, fmt)
    N, kw = _packed("wq", wq, ws, fmt)
    if kw != K:
        _fail(f"xq has {K} columns, wq {kw}")
    _scale("x_scale", x_scale, fmt)
    _scale("w_scale", w_scale, fmt)
    _device(xq, xs, wq, ws, x_scale, w_scale, out)
    if out is None:
        out = _empty((M, N), xq, stream, dtype or torch.bfloat16)
    else:
        _contiguous("out", out, (M, N), dtype)
    binding.sgq_fp4_gemm(xq, xs, x_scale, wq, ws, w_scale, out, M, N, K, f, _dtype(out), stream)
    return out
