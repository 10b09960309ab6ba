"""Latent attention without a GPU: what the C ABI and the helpers refuse, and the rotary table."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
from fp8_block_scaled_sgq_gb300 import binding, build

A, B, C, D, E, F, G = (0x10000 * i for i in range(1, 8))   # fake aligned addresses: never dereferenced
S = 1
INV, MIS, OK = binding.SGQ_ERR_INVALID_ARG, binding.SGQ_ERR_MISALIGNED, binding.SGQ_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def caller(f, names, defaults):
    def call(**k):
        assert not set(k) - set(names)
        return f(*[k.get(n, defaults[n]) for n in names], S)
    return call


def test_rotary_validation(lib):
    d = dict(x=A, T=4, H=2, D=192, xt=384, xh=192, pos=B, table=C, max_pos=10, R=64, offset=128, inter=1, inverse=0,
             dtype=0, y=D, yt=384, yh=192)
    f = caller(lib.sgq_rotary, list(d), d)
    for bad in (dict(T=-1), dict(H=-1), dict(D=0), dict(D=2056), dict(D=196), dict(R=0), dict(R=12), dict(inter=0, R=24),
                dict(offset=136), dict(offset=4), dict(offset=-8), dict(inter=2), dict(inverse=2), dict(dtype=2),
                dict(xt=381), dict(xh=-192), dict(yh=184), dict(yt=8), dict(max_pos=0), dict(x=None), dict(pos=None),
                dict(table=None), dict(y=None), dict(x=D, xt=768)):
        assert f(**bad) == INV, bad
    for bad in (dict(x=A + 8), dict(table=C + 4), dict(y=D + 2), dict(pos=B + 4)):
        assert f(**bad) == MIS, bad
    assert f(T=0, x=None, y=None) == OK and f(H=0, x=None) == OK


def test_append_validation(lib):
    d = dict(q=A, qt=3072, qh=192, k=B, kt=576, latent=C, lt=576, pos=D, slots=E, table=F, max_pos=10, T=4, H=16, L=512,
             R=64, inter=1, dtype=0, qo=G, qot=1024, qoh=64, ko=None, kot=0, cache=A + 64, pages=8, page=16, cp=9216,
             cr=576)
    f = caller(lib.sgq_latent_append, list(d), d)
    for bad in (dict(T=-1), dict(H=-1), dict(L=0), dict(L=20), dict(R=264), dict(R=4), dict(inter=3), dict(dtype=-1),
                dict(kt=577), dict(cr=568), dict(page=0), dict(pages=-1), dict(q=None), dict(qo=None), dict(k=None),
                dict(latent=None), dict(slots=None), dict(cache=None), dict(qoh=56), dict(q=G), dict(ko=A, kot=8)):
        assert f(**bad) == INV, bad
    for bad in (dict(q=A + 8), dict(latent=C + 2), dict(cache=A + 4), dict(slots=E + 4), dict(ko=A + 8, kot=64)):
        assert f(**bad) == MIS, bad
    assert f(T=0, k=None, cache=None) == OK


ATT = dict(q=A, qr=576, T=4, H=16, cache=B, pages=8, page=16, cp=9216, cr=576, L=512, R=64, table=C, width=2, B=4,
           lens=D, starts=None, scale=0.1, dtype=0, out=E, lse=None, ws=F, ws_bytes=1 << 40)


def test_attention_validation(lib):
    f = caller(lib.sgq_latent_attention, list(ATT), ATT)
    for bad in (dict(T=-1), dict(H=0), dict(H=65536), dict(T=1 << 27), dict(B=-1), dict(L=64), dict(L=640), dict(L=200),
                dict(R=0), dict(R=72), dict(R=12), dict(dtype=7), dict(qr=568), dict(qr=580), dict(cr=568),
                dict(cp=9208), dict(page=24), dict(page=0), dict(pages=0), dict(width=-1), dict(width=1 << 28),
                dict(T=5), dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(cache=None),
                dict(table=None), dict(lens=None), dict(out=None), dict(ws=None), dict(B=0, starts=G)):
        assert f(**bad) == INV, bad
    for bad in (dict(q=A + 8), dict(cache=B + 8), dict(out=E + 4), dict(ws=F + 4), dict(table=C + 2), dict(lens=D + 1),
                dict(starts=G + 2), dict(lse=G + 3)):
        assert f(**bad) == MIS, bad
    assert f(T=0, B=0, q=None, out=None, ws=None) == OK


def test_workspace_validation(lib):
    f = lib.sgq_latent_attention_workspace
    import ctypes
    n = ctypes.c_int64()
    assert f(4, 16, 512, None) == INV
    for bad in ((-1, 16, 512), (4, 0, 512), (4, 16, 100), (4, 16, 640), (4, 65536, 512)):
        assert f(*bad, ctypes.byref(n)) == INV, bad


def test_prefill_validation(lib):
    d = dict(q=A, qt=3072, qh=192, T=4, k=B, kt=4096, kh=256, kr=C, krt=64, v=D, vt=4096, vh=256, S=6, H=16, N=128, R=64,
             qs=E, ks=F, B=1, scale=0.1, causal=1, dtype=0, out=G, lse=None)
    f = caller(lib.sgq_latent_prefill, list(d), d)
    for bad in (dict(T=-1), dict(S=-1), dict(H=0), dict(N=96), dict(N=256), dict(R=0), dict(R=72), dict(R=20),
                dict(dtype=2), dict(causal=2), dict(qt=3073), dict(vh=-256), dict(krt=4), dict(krt=0), dict(kh=0), dict(qt=0), dict(vt=0), dict(B=0), dict(q=None),
                dict(k=None), dict(kr=None), dict(v=None), dict(qs=None), dict(ks=None), dict(out=None),
                dict(scale=float("inf")), dict(scale=-1.0)):
        assert f(**bad) == INV, bad
    for bad in (dict(q=A + 8), dict(k=B + 2), dict(kr=C + 8), dict(v=D + 8), dict(out=G + 8), dict(qs=E + 2),
                dict(ks=F + 1), dict(lse=A + 2)):
        assert f(**bad) == MIS, bad
    assert f(T=0, q=None, out=None) == OK


def test_helpers_refuse():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos, table = torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        sgq.rotary(x, pos, table)
    with pytest.raises(ValueError, match="bfloat16"):
        sgq.rotary(x.float(), pos, table)
    with pytest.raises(ValueError, match="positions"):
        sgq.rotary(x, pos.int(), table)
    with pytest.raises(ValueError, match="contiguous"):
        sgq.rotary(x.transpose(1, 2), pos, table)
    with pytest.raises(ValueError, match="T, H, D"):
        sgq.rotary(x[0], pos, table)
    kv, slots = torch.zeros(2, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    cache = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows of"):
        sgq.latent_append(None, kv[:, 512:], kv[:, :504], pos, slots, table, cache)
    with pytest.raises(ValueError, match="one element type"):
        sgq.latent_append(None, kv[:, 512:], kv[:, :512], pos, slots, table, cache.half())
    with pytest.raises(ValueError, match="without q_rot"):
        with pytest.MonkeyPatch.context() as m:
            m.setattr("fp8_block_scaled_sgq_gb300.latent._device", lambda *a: None)
            sgq.latent_append(None, kv[:, 512:], kv[:, :512], pos, slots, table, cache, q_out=x)
    q, pages, lens = torch.zeros(2, 16, 576, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="without q_starts"):
        sgq.latent_attention(q, cache, pages[:1], lens[:1], 0.1, 512)
    with pytest.raises(ValueError, match="kv_lens"):
        sgq.latent_attention(q, cache, pages, lens.long(), 0.1, 512)
    with pytest.raises(ValueError, match="evenly spaced"):
        sgq.latent_attention(torch.zeros(2, 32, 576, dtype=torch.bfloat16)[:, :16], cache, pages, lens, 0.1, 512)
    k = torch.zeros(5, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_rot"):
        sgq.latent_prefill(q[..., :192], k, kv[:, 512:], k, lens, lens, 0.1)


def test_rotary_table():
    t = sgq.rotary_table(1000, 64, device="cpu")
    assert t.shape == (1000, 64) and t.dtype == torch.float32
    for p, i in [(0, 0), (1, 0), (999, 0), (999, 31), (512, 7)]:
        a = p * 10000.0 ** (-2 * i / 64)
        assert t[p, i] == np.float32(math.cos(a)) and t[p, 32 + i] == np.float32(math.sin(a))
    # interpolated positions: position 4 p of the stretched table is position p of the plain one
    s = sgq.rotary_table(4000, 64, factor=4.0, device="cpu")
    assert torch.allclose(s[::4], t, atol=1e-6)
    # by parts: fast pairs keep their frequency, slow ones are interpolated, those between lie between
    y = sgq.rotary_table(4000, 64, factor=4.0, original_max=1000, attention_factor=1.25, device="cpu")
    plain = sgq.rotary_table(4000, 64, attention_factor=1.25, device="cpu")
    assert torch.equal(y[:, 0], plain[:, 0])
    assert torch.allclose(y[:, 31], s[:, 31] * 1.25, atol=1e-6)
    a, b, c = (math.atan2(v[10, 32 + 10], v[10, 10]) for v in (s, y, plain))
    assert min(a, c) <= b <= max(a, c)
    for bad in (dict(rot=63), dict(max_pos=0), dict(base=1.0), dict(factor=0.5)):
        with pytest.raises(ValueError):
            sgq.rotary_table(**{"max_pos": 10, "rot": 64, "device": "cpu", **bad})
