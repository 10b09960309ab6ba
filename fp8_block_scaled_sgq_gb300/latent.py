"""Latent attention and the steps around it, as functions of torch CUDA tensors.

These helpers check shapes, types and strides, allocate what they return (and
the attention's workspace) on the stream of the call, and call the binding; the
work is in ``libsgq.so`` (``include/sgq.h``, "Latent attention").  Tensors are
bfloat16 or float16, one type for a call.  Wrong shapes, types or strides raise
ValueError before anything is launched.
"""
from __future__ import annotations

import contextlib
import math

from . import binding


def _on(stream):
    """The allocations of a call belong to its stream, so that their memory is
    not handed out again while its kernels run."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _dtype(x, *others) -> int:
    import torch
    for t in others:
        if t is not None and t.dtype != x.dtype:
            raise ValueError(f"one element type a call: {x.dtype} and {t.dtype}")
    if x.dtype == torch.bfloat16:
        return binding.SGQ_BF16
    if x.dtype == torch.float16:
        return binding.SGQ_FP16
    raise ValueError(f"element type {x.dtype} is neither bfloat16 nor float16")


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _inner(name: str, t):
    _need(t.shape[-1] <= 1 or t.stride(-1) == 1, f"{name}: the last dimension is not contiguous")
    return t


def _index(name: str, t, dtype, n: int):
    """A whole-number tensor of the given type with n contiguous entries."""
    _need(t.dtype == dtype and t.dim() == 1 and t.shape[0] == n and t.is_contiguous(),
          f"{name}: expected {n} contiguous {dtype} entries, got {tuple(t.shape)} of {t.dtype}")
    return t


def _device(x, *others):
    _need(x.is_cuda, "the tensors are not on a CUDA device")
    for t in others:
        _need(t is None or t.device == x.device, "the tensors are on different devices")


def rotary_table(max_pos: int, rot: int, base: float = 10000.0, factor: float = 1.0, original_max: int = 0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, attention_factor: float = 1.0, device="cuda"):
    """fp32 [max_pos, rot]: rot/2 cosines, then rot/2 sines, of each position's angles.

    Pair i turns by base^(-2i/rot) a position.  ``factor`` > 1 stretches the
    context: with ``original_max`` = 0 every frequency is divided by it
    (positions interpolated); with the trained length in ``original_max``,
    pairs that turn more than ``beta_fast`` times over it keep their frequency,
    pairs that turn less than ``beta_slow`` times are divided by ``factor``, and
    those between are blended linearly in the pair's index.
    ``attention_factor`` multiplies cosines and sines.  Angles are computed in
    64 bits, once, when the table is made.
    """
    import torch
    _need(max_pos > 0 and rot > 0 and rot % 2 == 0, "max_pos and an even rot are needed")
    _need(base > 1.0 and factor >= 1.0, "base > 1 and factor >= 1 are needed")
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    freq = base ** (-2.0 * i / rot)
    if factor > 1.0:
        keep = torch.zeros_like(freq)
        if original_max > 0:
            def pair_of(turns):   # the pair that turns so many times over the trained length
                return rot * math.log(original_max / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
            lo, hi = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rot // 2 - 1)
            keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return (torch.cat([angle.cos(), angle.sin()], dim=1) * attention_factor).float()


def _table(table):
    import torch
    _need(table.dim() == 2 and table.dtype == torch.float32 and table.is_contiguous(),
          "table: expected a contiguous float32 [max_pos, rot] tensor")
    return table


def rotary(x, positions, table, offset: int = 0, interleaved: bool = True, inverse: bool = False, out=None,
           stream=None):
    """x [T, H, D] with elements [offset, offset + rot) of every head rotated by its token's position.

    positions: int64 [T]; table: ``rotary_table``.  interleaved: pairs (2i, 2i + 1), else (i, i + rot/2).
    inverse: rotate back, which is also the gradient.  out may be x (in place); returns out.
    """
    import torch
    _need(x.dim() == 3, f"x: expected [T, H, D], got {tuple(x.shape)}")
    dt = _dtype(x, out)
    T, H, D = _inner("x", x).shape
    _index("positions", positions, torch.int64, T)
    max_pos, R = _table(table).shape
    _device(x, positions, table, out)
    if out is None:
        with _on(stream):
            out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    _need(out.shape == x.shape, "out: not of x's shape")
    _inner("out", out)
    binding.sgq_rotary(x, T, H, D, x.stride(0), x.stride(1), positions, table, max_pos, R, offset, interleaved, inverse,
                       dt, out, out.stride(0), out.stride(1), stream)
    return out


def _cache(cache):
    _need(cache.dim() == 3, f"cache: expected [pages, page, width], got {tuple(cache.shape)}")
    return _inner("cache", cache)


def latent_append(q_rot, k_rot, latent, positions, slots, table, cache, interleaved: bool = True, q_out=None,
                  k_out=None, stream=None):
    """Rotates queries and keys and writes the tokens' rows [latent | rotated key] into the paged cache, in one launch.

    q_rot: the queries' positional parts [T, H, R], or None; k_rot [T, R]; latent [T, L]; positions, slots: int64 [T]
    (slot = page number * page size + row; negative: padding, no row); cache [pages, page, L + R].  Returns the rotated
    queries: q_out (which may be q_rot, or a view of the attention's query tensor) or a new tensor.  k_out, if given,
    receives the rotated keys.
    """
    import torch
    T, R = _inner("k_rot", k_rot).shape
    L = _inner("latent", latent).shape[1]
    dt = _dtype(k_rot, q_rot, latent, cache, q_out, k_out)
    _need(latent.shape[0] == T, "latent: not one row a token")
    _index("positions", positions, torch.int64, T)
    _index("slots", slots, torch.int64, T)
    max_pos = _table(table).shape[0]
    _need(table.shape[1] == R, "table: not of the rotated width")
    pages, page, width = _cache(cache).shape
    _need(width == L + R, f"cache: rows of {width}, not {L} + {R}")
    _device(k_rot, q_rot, latent, positions, slots, table, cache, q_out, k_out)
    H, qs, qo = 0, (0, 0), (0, 0)
    if q_rot is not None:
        _need(q_rot.dim() == 3 and q_rot.shape[0] == T and q_rot.shape[2] == R, "q_rot: expected [T, H, R]")
        H = _inner("q_rot", q_rot).shape[1]
        if q_out is None:
            with _on(stream):
                q_out = torch.empty((T, H, R), dtype=q_rot.dtype, device=q_rot.device)
        _need(q_out.shape == q_rot.shape, "q_out: not of q_rot's shape")
        _inner("q_out", q_out)
        qs, qo = (q_rot.stride(0), q_rot.stride(1)), (q_out.stride(0), q_out.stride(1))
    else:
        _need(q_out is None, "q_out without q_rot")
    if k_out is not None:
        _need(k_out.shape == k_rot.shape, "k_out: not of k_rot's shape")
        _inner("k_out", k_out)
    binding.sgq_latent_append(q_rot, qs[0], qs[1], k_rot, k_rot.stride(0), latent, latent.stride(0), positions, slots,
                              table, max_pos, T, H, L, R, interleaved, dt, q_out, qo[0], qo[1], k_out,
                              k_out.stride(0) if k_out is not None else 0, cache, pages, page, cache.stride(0),
                              cache.stride(1), stream)
    return q_out


def latent_attention(q, cache, page_table, kv_lens, scale: float, latent: int, q_starts=None, out=None, lse=None,
                     workspace=None, stream=None):
    """Absorbed latent attention over a paged cache: out [T, H, latent].

    q [T, H, latent + R]; cache [pages, page, latent + R]; page_table int32 [B, width]; kv_lens int32 [B]: rows of each
    request, its query tokens' own rows last.  q_starts int32 [B + 1]: the requests' first query tokens (a chunk sees
    its own tokens causally); None: one token a request.  lse: fp32 [T, H] to receive the logarithm of the softmax
    sums.  workspace: ``sgq_latent_attention_workspace`` bytes of this device's memory that no call running at the
    same time uses; None: allocated here.
    """
    import torch
    _need(q.dim() == 3, f"q: expected [T, H, latent + R], got {tuple(q.shape)}")
    dt = _dtype(q, cache, out)
    T, H, W = _inner("q", q).shape
    pages, page, width = _cache(cache).shape
    _need(width == W, f"cache: rows of {width}, queries of {W}")
    _need(T <= 1 or H == 1 or q.stride(0) == H * q.stride(1), "q: tokens and heads are not evenly spaced rows")
    row = q.stride(1) if H > 1 else q.stride(0) if T > 1 else W
    _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.is_contiguous(),
          "page_table: expected a contiguous int32 [B, width] tensor")
    B = page_table.shape[0]
    _index("kv_lens", kv_lens, torch.int32, B)
    if q_starts is not None:
        _index("q_starts", q_starts, torch.int32, B + 1)
    else:
        _need(T == B, f"{T} query tokens for {B} requests, without q_starts")
    _device(q, cache, page_table, kv_lens, q_starts, out, lse, workspace)
    with _on(stream):
        if out is None:
            out = torch.empty((T, H, latent), dtype=q.dtype, device=q.device)
        if workspace is None:
            workspace = torch.empty(binding.sgq_latent_attention_workspace(T, H, latent), dtype=torch.uint8,
                                    device=q.device)
    _need(out.shape == (T, H, latent) and out.is_contiguous(), "out: expected a contiguous [T, H, latent] tensor")
    _need(lse is None or (lse.shape == (T, H) and lse.dtype == torch.float32 and lse.is_contiguous()),
          "lse: expected a contiguous float32 [T, H] tensor")
    binding.sgq_latent_attention(q, row, T, H, cache, pages, page, cache.stride(0), cache.stride(1), latent, W - latent,
                                 page_table, page_table.shape[1], B, kv_lens, q_starts, scale, dt, out, lse, workspace,
                                 workspace.numel() * workspace.element_size(), stream)
    return out


def latent_prefill(q, k, k_rot, v, q_starts, kv_starts, scale: float, causal: bool = True, out=None, lse=None,
                   stream=None):
    """Expanded latent attention of ragged prompts: out [T, H, N].

    q [T, H, N + R]; k, v [S, H, N]; k_rot [S, R], shared by the heads; q_starts, kv_starts int32 [B + 1].  causal: the
    last query of a request sees all its keys, each one before it one key less.  lse: fp32 [T, H] to receive the
    logarithm of the softmax sums.
    """
    import torch
    _need(q.dim() == 3 and k.dim() == 3 and v.dim() == 3 and k_rot.dim() == 2, "expected q, k, v of 3 dimensions, k_rot of 2")
    dt = _dtype(q, k, k_rot, v, out)
    T, H, W = _inner("q", q).shape
    S, _, N = _inner("k", k).shape
    _need(k.shape == (S, H, N) and v.shape == (S, H, N), "k, v: expected [S, H, N] with q's heads")
    R = W - N
    _need(k_rot.shape == (S, R), f"k_rot: expected [{S}, {R}]")
    _inner("k_rot", k_rot), _inner("v", v)
    B = q_starts.shape[0] - 1
    _index("q_starts", q_starts, torch.int32, B + 1)
    _index("kv_starts", kv_starts, torch.int32, B + 1)
    _device(q, k, k_rot, v, q_starts, kv_starts, out, lse)
    if out is None:
        with _on(stream):
            out = torch.empty((T, H, N), dtype=q.dtype, device=q.device)
    _need(out.shape == (T, H, N) and out.is_contiguous(), "out: expected a contiguous [T, H, N] tensor")
    _need(lse is None or (lse.shape == (T, H) and lse.dtype == torch.float32 and lse.is_contiguous()),
          "lse: expected a contiguous float32 [T, H] tensor")
    binding.sgq_latent_prefill(q, q.stride(0), q.stride(1), T, k, k.stride(0), k.stride(1), k_rot, k_rot.stride(0), v,
                               v.stride(0), v.stride(1), S, H, N, R, q_starts, kv_starts, B, scale, causal, dt, out,
                               lse, stream)
    return out
