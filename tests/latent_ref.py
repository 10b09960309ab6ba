"""Definitions of the latent-attention operators in 64 bits, on the CPU, and the error bounds the tests hold them to.

Bounds, fixed from the number formats: u is the unit roundoff of the element type (2^-8 bf16, 2^-11 fp16).  A result
is rounded once (u |ref|).  Softmax weights are rounded once as a product's operand, which moves a row by at most
u sum_j w_j |v_j|.  A score of W products is off by at most e = W 2^-23 scale sum |q c| (fp32 accumulation, truncating),
which moves weights relatively by 2 e; exp2 and the sums add less than 2^-20.
"""
import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return t.detach().double().cpu().numpy()


def rotate(x, positions, table, offset, interleaved, inverse=False):
    """x [T, H, D] (numpy, 64 bits) -> (rotated, bound's magnitude |a c| + |b s|)."""
    y, mag = x.copy(), np.zeros_like(x)
    R = table.shape[1]
    c, s = table[positions, :R // 2][:, None], table[positions, R // 2:][:, None]
    if inverse:
        s = -s
    i = np.arange(R // 2)
    ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + R // 2 + i)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def check_rotation(got, ref, mag, dtype):
    tol = UNIT[dtype] * np.abs(ref) + 2.0 ** -22 * mag + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), f"off by {(err - tol).max()} past the bound"


def attend(q, k, v, visible, scale):
    """q [n, W], k [m, W], v [m, N], visible [n, m] -> (out, lse, sum w |v|, score error bound) of every row."""
    s = (q @ k.T) * scale
    s[~visible] = -np.inf
    alive = visible.any(axis=1)
    top = np.where(alive, s.max(axis=1, initial=-np.inf), 0.0)
    p = np.where(visible, np.exp(s - top[:, None]), 0.0)
    total = p.sum(axis=1)
    w = p / np.where(alive, total, 1.0)[:, None]
    lse = np.where(alive, top + np.log(np.where(alive, total, 1.0)), -np.inf)
    mags = (np.abs(q) @ np.abs(k).T) * abs(scale)
    e = q.shape[1] * 2.0 ** -23 * np.where(visible, mags, 0.0).max(axis=1, initial=0.0)
    return w @ v, lse, w @ np.abs(v), e


def check_rows(got, got_lse, ref, lse, mag, e, dtype, what=""):
    u = UNIT[dtype]
    got = f64(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    tol = u * np.abs(ref) + (u + 2 * e[:, None] + 2.0 ** -20) * mag + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = np.abs(got - ref)
    if not (err <= tol).all():
        at = np.unravel_index(np.argmax(err - tol), err.shape)
        raise AssertionError(f"{what}: {(err > tol).sum()} of {err.size} past the bound, worst at {at}: "
                             f"got {got[at]}, want {ref[at]} within {tol[at]}")
    if got_lse is not None:
        got_lse = f64(got_lse)
        none = np.isneginf(lse)
        assert (np.isneginf(got_lse) == none).all(), f"{what}: empty rows"
        bad = np.abs(got_lse[~none] - lse[~none]) > (e[~none] + 2.0 ** -18 + 2.0 ** -21 * np.abs(lse[~none]))
        assert not bad.any(), f"{what}: logarithms of {bad.sum()} rows"
