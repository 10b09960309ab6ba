"""Latent attention and the steps around it, as functions of torch CUDA tensors.

These helpers check shapes, types and strides, allocate what they return (and
the attention's workspace) on the stream of the call, and call the binding; the
work is in ``libsgq.so`` (``include/sgq.h``, "Latent attention").  Tensors are
bfloat16 or float16, one type for a call, on the current device.  Wrong shapes,
types or strides raise ValueError before anything is launched, and so does a
tensor that requires a gradient while gradients are recorded: none is here.
"""
from __future__ import annotations

import functools
import math

from . import binding


def _empty(shape, like, stream):
    """A new tensor of like's type and device that belongs to the call's stream,
    so that its memory is not handed out again while its kernels run."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if isinstance(stream, int):   # (0 is the default stream's handle; torch makes a new stream of ExternalStream(0))
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=like.dtype, device=like.device)


# The checks below run on every call of a decode step: plain comparisons, the
# message made only when one fails.

def _dtype(x, *others) -> int:
    import torch
    dt, graded = x.dtype, torch.is_grad_enabled()
    if graded and x.requires_grad:
        _graded()
    for t in others:
        if t is not None:
            if t.dtype != dt:
                raise ValueError(f"one element type a call: {dt} and {t.dtype}")
            if graded and t.requires_grad:
                _graded()
    if dt == torch.bfloat16:
        return binding.SGQ_BF16
    if dt == torch.float16:
        return binding.SGQ_FP16
    raise ValueError(f"element type {dt} is neither bfloat16 nor float16")


def _fail(what: str):
    raise ValueError(what)


def _graded():
    _fail("a tensor requires a gradient, and none is recorded here: detach it, or call under torch.no_grad() "
          "(rotary's gradient is rotary with inverse=True)")


def _strides(name: str, t, dims: int):
    """t's strides but the last, which has to be 1."""
    s = t.stride()
    if len(s) != dims:
        _fail(f"{name}: expected {dims} dimensions, got {tuple(t.shape)}")
    if s[-1] != 1 and t.shape[-1] > 1:
        _fail(f"{name}: the last dimension is not contiguous")
    return s[:-1]


def _index(name: str, t, dtype, n: int):
    """A whole-number tensor of the given type with n contiguous entries."""
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        _fail(f"{name}: expected {n} contiguous {dtype} entries, got {tuple(t.shape)} of {t.dtype}")


def _device(x, *others) -> int:
    """The index of the tensors' device, which is the current one: stream, workspace and launch are its own."""
    import torch
    if not x.is_cuda:
        _fail("the tensors are not on a CUDA device")
    at = x.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            _fail("the tensors are on different devices")
    if at != torch.cuda.current_device():
        _fail(f"the tensors are on device {at}, the current one is {torch.cuda.current_device()}")
    return at


def _contiguous(name: str, t, shape, dtype=None):
    if t.shape != shape or not t.is_contiguous() or (dtype is not None and t.dtype != dtype):
        _fail(f"{name}: expected a contiguous {tuple(shape)} tensor{'' if dtype is None else f' of {dtype}'}")


def rotary_table(max_pos: int, rot: int, base: float = 10000.0, factor: float = 1.0, original_max: int = 0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, attention_factor: float = 1.0, device="cuda"):
    """fp32 [max_pos, rot]: rot/2 cosines, then rot/2 sines, of each position's angles.

    Pair i turns by base^(-2i/rot) a position.  ``factor`` > 1 stretches the
    context: with ``original_max`` = 0 every frequency is divided by it
    (positions interpolated); with the trained length in ``original_max``,
    pairs that turn more than ``beta_fast`` times over it keep their frequency,
    pairs that turn less than ``beta_slow`` times are divided by ``factor``, and
    those between are blended linearly in the pair's index (the two bounds
    rounded outwards to whole pairs).
    ``attention_factor`` multiplies cosines and sines.  Angles are computed in
    64 bits, once, when the table is made.
    """
    import torch
    if max_pos <= 0 or rot <= 0 or rot % 2 != 0:
        _fail("max_pos > 0 and an even rot > 0 are needed")
    if base <= 1.0 or factor < 1.0:
        _fail("base > 1 and factor >= 1 are needed")
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    freq = base ** (-2.0 * i / rot)
    if factor > 1.0:
        keep = torch.zeros_like(freq)
        if original_max > 0:
            def pair_of(turns):   # the pair that turns so many times over the trained length
                return rot * math.log(original_max / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
            # The blend's end may lie past the last pair (all pairs turn more than beta_slow times over a long trained
            # length) or before the first one (none does); its start is the first pair at the earliest.
            lo, hi = max(math.floor(pair_of(beta_fast)), 0), math.ceil(pair_of(beta_slow))
            if hi > 0:
                keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return (torch.cat([angle.cos(), angle.sin()], dim=1) * attention_factor).float()


def _table(table):
    import torch
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        _fail("table: expected a contiguous float32 [max_pos, rot] tensor")
    return table.shape


def rotary(x, positions, table, offset: int = 0, interleaved: bool = True, inverse: bool = False, out=None,
           stream=None):
    """x [T, H, D] with elements [offset, offset + rot) of every head rotated by its token's position.

    positions: int64 [T]; table: ``rotary_table``.  interleaved: pairs (2i, 2i + 1), else (i, i + rot/2).
    inverse: the transpose, i.e. the gradient; it rotates back where the table's ``attention_factor`` is 1 (else x comes
    back times its square).  out may be x (in place); returns out.
    """
    import torch
    dt = _dtype(x, out)
    if x.dim() != 3:
        _fail(f"x: expected [T, H, D], got {tuple(x.shape)}")
    T, H, D = x.shape
    xt, xh = _strides("x", x, 3)
    _index("positions", positions, torch.int64, T)
    max_pos, R = _table(table)
    _device(x, positions, table, out)
    if out is None:
        out = _empty((T, H, D), x, stream)
    elif out.shape != x.shape:
        _fail("out: not of x's shape")
    yt, yh = _strides("out", out, 3)
    binding.sgq_rotary(x, T, H, D, xt, xh, positions, table, max_pos, R, offset, interleaved, inverse, dt, out, yt, yh,
                       stream)
    return out


def latent_append(q_rot, k_rot, latent, positions, slots, table, cache, interleaved: bool = True, q_out=None,
                  k_out=None, stream=None):
    """Rotates queries and keys and writes the tokens' rows [latent | rotated key] into the paged cache, in one launch.

    q_rot: the queries' positional parts [T, H, R], or None; k_rot [T, R]; latent [T, L]; positions, slots: int64 [T]
    (slot = page number * page size + row; negative: padding, no row); cache [pages, page, L + R].  Returns the rotated
    queries: q_out (which may be q_rot, or a view of the attention's query tensor) or a new tensor.  k_out, if given,
    receives the rotated keys.
    """
    import torch
    dt = _dtype(k_rot, q_rot, latent, cache, q_out, k_out)
    (kt,), (lt,), (cp, cr) = _strides("k_rot", k_rot, 2), _strides("latent", latent, 2), _strides("cache", cache, 3)
    T, R = k_rot.shape
    L = latent.shape[1]
    if latent.shape[0] != T:
        _fail("latent: not one row a token")
    _index("positions", positions, torch.int64, T)
    _index("slots", slots, torch.int64, T)
    max_pos, rot = _table(table)
    if rot != R:
        _fail("table: not of the rotated width")
    pages, page, width = cache.shape
    if width != L + R:
        _fail(f"cache: rows of {width}, not {L} + {R}")
    _device(k_rot, q_rot, latent, positions, slots, table, cache, q_out, k_out)
    H = qt = qh = ot = oh = ko = 0
    if q_rot is not None:
        qt, qh = _strides("q_rot", q_rot, 3)
        H = q_rot.shape[1]
        if q_rot.shape[0] != T or q_rot.shape[2] != R:
            _fail("q_rot: expected [T, H, R]")
        if q_out is None:
            q_out = _empty((T, H, R), q_rot, stream)
        elif q_out.shape != q_rot.shape:
            _fail("q_out: not of q_rot's shape")
        ot, oh = _strides("q_out", q_out, 3)
    elif q_out is not None:
        _fail("q_out without q_rot")
    if k_out is not None:
        if k_out.shape != k_rot.shape:
            _fail("k_out: not of k_rot's shape")
        ko, = _strides("k_out", k_out, 2)
    binding.sgq_latent_append(q_rot, qt, qh, k_rot, kt, latent, lt, positions, slots, table, max_pos, T, H, L, R,
                              interleaved, dt, q_out, ot, oh, k_out, ko, cache, pages, page, cp, cr, stream)
    return q_out


@functools.lru_cache(maxsize=256)
def _workspace_bytes(T: int, H: int, latent: int, device: int) -> int:
    """(of the current device, which is the last argument: sizes go by its number of SMs)"""
    return binding.sgq_latent_attention_workspace(T, H, latent)


def latent_attention(q, cache, page_table, kv_lens, scale: float, latent: int, q_starts=None, out=None, lse=None,
                     workspace=None, stream=None):
    """Absorbed latent attention over a paged cache: out [T, H, latent].

    q [T, H, latent + R]; cache [pages, page, latent + R]; page_table int32 [B, width]; kv_lens int32 [B]: rows of each
    request, its query tokens' own rows last.  q_starts int32 [B + 1]: the requests' first query tokens (a chunk sees
    its own tokens causally); None: one token a request.  lse: fp32 [T, H] to receive the logarithm of the softmax
    sums.  workspace: a contiguous tensor of ``sgq_latent_attention_workspace`` bytes that no call running at
    the same time uses; None: allocated here.
    """
    import torch
    dt = _dtype(q, cache, out)
    (qt, qh), (cp, cr) = _strides("q", q, 3), _strides("cache", cache, 3)
    T, H, W = q.shape
    pages, page, width = cache.shape
    if width != W:
        _fail(f"cache: rows of {width}, queries of {W}")
    if T > 1 and H > 1 and qt != H * qh:
        _fail("q: tokens and heads are not evenly spaced rows")
    row = qh if H > 1 else qt if T > 1 else W
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_contiguous():
        _fail("page_table: expected a contiguous int32 [B, width] tensor")
    B, table_width = page_table.shape
    _index("kv_lens", kv_lens, torch.int32, B)
    if q_starts is not None:
        _index("q_starts", q_starts, torch.int32, B + 1)
    elif T != B:
        _fail(f"{T} query tokens for {B} requests, without q_starts")
    device = _device(q, cache, page_table, kv_lens, q_starts, out, lse, workspace)
    if out is None:
        out = _empty((T, H, latent), q, stream)
    else:
        _contiguous("out", out, (T, H, latent))
    if lse is not None:
        _contiguous("lse", lse, (T, H), torch.float32)
    stream, own = binding._stream(stream), None
    if workspace is None:
        # Memory of torch's allocator without a tensor around it; it belongs to the call's stream, and goes back to
        # that stream's memory as soon as the call is queued.
        nbytes = _workspace_bytes(T, H, latent, device)
        workspace = own = torch.cuda.caching_allocator_alloc(nbytes, device, stream)
    else:
        if not workspace.is_contiguous():
            _fail("workspace: not contiguous")
        nbytes = workspace.numel() * workspace.element_size()
    try:
        binding.sgq_latent_attention(q, row, T, H, cache, pages, page, cp, cr, latent, W - latent, page_table,
                                     table_width, B, kv_lens, q_starts, scale, dt, out, lse, workspace, nbytes, stream)
    finally:
        if own is not None:
            torch.cuda.caching_allocator_delete(own)
    return out


def latent_prefill(q, k, k_rot, v, q_starts, kv_starts, scale: float, causal: bool = True, out=None, lse=None,
                   stream=None):
    """Expanded latent attention of ragged prompts: out [T, H, N].

    q [T, H, N + R]; k, v [S, H, N]; k_rot [S, R], shared by the heads; q_starts, kv_starts int32 [B + 1].  causal: the
    last query of a request sees all its keys, each one before it one key less.  lse: fp32 [T, H] to receive the
    logarithm of the softmax sums.
    """
    import torch
    dt = _dtype(q, k, k_rot, v, out)
    (qt, qh), (kt, kh), (vt, vh) = _strides("q", q, 3), _strides("k", k, 3), _strides("v", v, 3)
    rt, = _strides("k_rot", k_rot, 2)
    T, H, W = q.shape
    S, _, N = k.shape
    R = W - N
    if k.shape[1] != H or v.shape != k.shape:
        _fail("k, v: expected [S, H, N] with q's heads")
    if k_rot.shape[0] != S or k_rot.shape[1] != R:
        _fail(f"k_rot: expected [{S}, {R}]")
    B = q_starts.shape[0] - 1
    _index("q_starts", q_starts, torch.int32, B + 1)
    _index("kv_starts", kv_starts, torch.int32, B + 1)
    _device(q, k, k_rot, v, q_starts, kv_starts, out, lse)
    if out is None:
        out = _empty((T, H, N), q, stream)
    else:
        _contiguous("out", out, (T, H, N))
    if lse is not None:
        _contiguous("lse", lse, (T, H), torch.float32)
    binding.sgq_latent_prefill(q, qt, qh, T, k, kt, kh, k_rot, rt, v, vt, vh, S, H, N, R, q_starts, kv_starts, B, scale,
                               causal, dt, out, lse, stream)
    return out
