"""Definitions of the 4-bit linears' operators and of the norms on the CPU, and the error bounds the tests hold them to.

Quantisation is a rule of fp32 operations, written here with numpy's (IEEE), so codes and scale bytes are equal.  Where
its input is itself a computed fp32 value (silu, a norm) that is off by at most d relative to its 64-bit value, a scale byte
is one of those that amax (1 - d) and amax (1 + d) get, and a code's value is off by at most half a step at its place plus
d |x| / s.

An MMA adds the products of a group exactly (multiples of 1/4 up to 36, 16 or 32 of them), and groups in fp32, each addition
off by at most 2^-23 of the magnitudes it adds (truncation): K/16 additions are off by K/16 2^-23 sum |a||w|.
"""
import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
GROUP = {"mxfp4": 32, "nvfp4": 16}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)) for e in range(16) for f in range(8)][:127])


def f64(t):
    return t.detach().double().cpu().numpy()


def nearest(x, table):
    """Index of the entry of a rising table of magnitudes nearest to |x| (x within it), ties to the even index."""
    a = np.abs(x)
    mid = (table[1:] + table[:-1]) / 2
    low, high = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    return np.where(low % 2 == 0, low, high)


def scale_bytes(amax, fmt, t=1.0):
    """Scale bytes of groups with these largest magnitudes (fp32), and what their values are divided by (fp32)."""
    amax, t = amax.astype(np.float32), np.float32(t)
    if fmt == "mxfp4":
        s = np.maximum(amax, np.float32(1e-10)) / np.float32(6)
        half, e = np.frexp(s)
        byte = (e + 126 + (half > 0.5)).astype(np.uint8)
        return byte, np.ldexp(np.float32(1), byte.astype(np.int32) - 127).astype(np.float32)
    with np.errstate(over="ignore"):
        s = np.minimum(amax / (np.float32(6) * t), np.float32(448))
    byte = np.maximum(nearest(s.astype(np.float64), E4M3), 1).astype(np.uint8)
    return byte, (E4M3[byte].astype(np.float32) * t).astype(np.float32)


def quantise(x, fmt, t=1.0):
    """x [M, K] (values of 16-bit type) -> (nibbles [M, K], scale bytes [M, K/g])."""
    x = x.astype(np.float32)
    part = x.reshape(x.shape[0], -1, GROUP[fmt])
    bad = ~np.isfinite(part).all(axis=-1)
    part = np.where(bad[..., None], np.float32(0), part)
    byte, d = scale_bytes(np.abs(part).max(axis=-1), fmt, t)
    none = (bad | (d == 0))[..., None]       # (a product s t below fp32's smallest value stands for zeros, whatever the codes)
    with np.errstate(over="ignore"):
        q = np.where(none, 0, part) / np.where(none, 1, d[..., None])
    nib = nearest(np.minimum(np.abs(q), 6).astype(np.float64), LEVELS) + 8 * np.signbit(part)
    nib = np.where(none, 0, nib)
    byte = np.where(bad, 255 if fmt == "mxfp4" else 0x7F, byte)
    return nib.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def values(nib, byte, fmt, t=1.0):
    """What nibbles and scale bytes stand for, in 64 bits (s t rounded to fp32, as the rule has it)."""
    if fmt == "mxfp4":
        s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    else:
        s = np.where(byte >= 127, np.nan, E4M3[np.minimum(byte, 126)])
        s = (s.astype(np.float32) * np.float32(t)).astype(np.float64)
    v = LEVELS[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    return (v.reshape(byte.shape[0], -1, GROUP[fmt]) * s[..., None]).reshape(nib.shape)


def pack(nib):
    return (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    q = q.detach().cpu().numpy()
    return np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1)


def to_tiles(byte, fill=0):
    """Scale bytes [M, G] -> tiles [ceil(M/128), ceil(G/4), 512], byte by byte from the definition; rows past M hold `fill`."""
    M, G = byte.shape
    out = np.full((-(-M // 128), -(-G // 4), 512), fill, np.uint8)
    for j in range(out.shape[1] * 4):
        r = np.arange(M)
        out[r // 128, j // 4, r % 32 * 16 + r % 128 // 32 * 4 + j % 4] = byte[:, j] if j < G else 0
    return out


def from_tiles(tiles, M, G):
    t = tiles.detach().cpu().numpy()
    r, j = np.arange(M)[:, None], np.arange(G)[None]
    return t[r // 128, j // 4, r % 32 * 16 + r % 128 // 32 * 4 + j % 4]


def check_codes(nib, byte, x, fmt, t, d, what=""):
    """nib, byte: what quantisation made of values that are off by at most d (relative) from x (64 bits)."""
    g = GROUP[fmt]
    part = x.reshape(x.shape[0], -1, g)
    amax = np.abs(part).max(axis=-1)
    lo, hi = scale_bytes(amax * (1 - d), fmt, t)[0], scale_bytes(amax * (1 + d), fmt, t)[0]
    assert ((byte >= lo) & (byte <= hi)).all(), f"{what}: scale bytes"
    s = values(np.full_like(nib, 2), byte, fmt, t)      # a code's step is in units of s
    assert (nib[s == 0] == 0).all(), f"{what}: codes under scales of zero"
    q, v = np.where(s == 0, 0, np.abs(x)) / np.where(s == 0, 1, s), LEVELS[nib & 7]
    up, down = np.append(LEVELS, 9.0)[(nib & 7) + 1], LEVELS[np.maximum((nib & 7).astype(int) - 1, 0)]
    slack = d * q + 2.0 ** -22 * q
    assert (np.where(v < 6, q <= (v + up) / 2 + slack, True)).all() and (q >= np.where(v > 0, (v + down) / 2, 0) - slack).all(), \
        f"{what}: codes"
    sure = q > 0.26
    assert ((nib >= 8) == (x < 0))[sure].all(), f"{what}: signs"


def check_product(d, a, w, alpha, dtype, what=""):
    """d against a w^T alpha (a, w: 64-bit values)."""
    ref = a @ w.T * alpha
    mag = np.abs(a) @ np.abs(w).T * abs(alpha)
    tol = UNIT[dtype] * np.abs(ref) + (a.shape[1] / 16 * 2.0 ** -23 + 2.0 ** -22) * mag
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    got = f64(d)
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: not finite"
    bad = err > tol
    if bad.any():
        at = np.unravel_index(np.argmax(err - tol), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} past the bound, first rows {np.unique(np.argwhere(bad)[:, 0])[:8]}, "
                             f"worst at {at}: got {got[at]}, want {ref[at]} within {tol[at]}")


# A row's mean square: at most 64 additions one after the other (32 squares a thread, 10 exchanges, and the products' own
# roundings), each off by 2^-24, halved by the root; 8 more roundings up to the value: 40 2^-24 < 2^-18.
NORM = 2.0 ** -18


def norm(x, weight, eps, offset):
    return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps) * (weight + offset)
