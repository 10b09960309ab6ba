"""4-bit linears and norms without a GPU: what the C ABI and the helpers refuse, and the layout of scales."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
from fp8_block_scaled_sgq_gb300 import binding, build, fp4, norms
import fp4_ref as ref

A, B, C, D, E, F, G, H = (0x10000 * i for i in range(1, 9))   # fake aligned addresses: never dereferenced
S = 1
INV, MIS, OK = binding.SGQ_ERR_INVALID_ARG, binding.SGQ_ERR_MISALIGNED, binding.SGQ_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def caller(f, defaults):
    def call(**k):
        assert not set(k) - set(defaults)
        return f(*[k.get(n, v) for n, v in defaults.items()], S)
    return call


def test_quant_validation(lib):
    f = caller(lib.sgq_quant_fp4, dict(x=A, M=4, K=64, stride=64, fmt=1, t=B, silu=0, dtype=0, xq=C, xs=D))
    for bad in (dict(M=-1), dict(K=0), dict(K=48), dict(fmt=2), dict(fmt=0), dict(silu=2), dict(dtype=2), dict(stride=56),
                dict(stride=65), dict(silu=1), dict(x=None), dict(xq=None), dict(xs=None), dict(M=1 << 31),
                dict(M=1 << 30, K=2048, stride=2048)):
        assert f(**bad) == INV, bad
    for bad in (dict(x=A + 8), dict(xq=C + 4), dict(xs=D + 8), dict(t=B + 2)):
        assert f(**bad) == MIS, bad
    assert f(M=0, x=None, xq=None, xs=None) == OK


def test_dequant_validation(lib):
    f = caller(lib.sgq_dequant_fp4, dict(xq=A, xs=B, M=4, K=64, fmt=0, t=None, dtype=1, y=C))
    for bad in (dict(M=-1), dict(K=40), dict(fmt=-1), dict(t=D), dict(dtype=3), dict(xq=None), dict(xs=None), dict(y=None)):
        assert f(**bad) == INV, bad
    for bad in (dict(xq=A + 8), dict(xs=B + 1), dict(y=C + 2)):
        assert f(**bad) == MIS, bad
    assert f(M=0, xq=None, y=None) == OK


def test_gemm_validation(lib):
    f = caller(lib.sgq_fp4_gemm, dict(aq=A, as_=B, at=G, wq=C, ws=D, wt=H, d=E, M=4, N=16, K=64, fmt=1, dtype=0))
    for bad in (dict(M=-1), dict(N=0), dict(N=12), dict(K=16), dict(K=0), dict(fmt=0), dict(fmt=0, at=None), dict(fmt=3),
                dict(dtype=-1), dict(aq=None), dict(as_=None), dict(wq=None), dict(ws=None), dict(d=None), dict(N=1 << 31),
                dict(M=1 << 31), dict(M=(1 << 31) - 1024), dict(N=(1 << 31) - 1024), dict(K=(1 << 26) + 64)):
        assert f(**bad) == INV, bad
    for bad in (dict(aq=A + 8), dict(as_=B + 8), dict(wq=C + 2), dict(ws=D + 4), dict(d=E + 8), dict(at=G + 2), dict(wt=H + 1)):
        assert f(**bad) == MIS, bad
    assert f(M=0, aq=None, d=None) == OK


def test_norm_validation(lib):
    d = dict(x=A, xt=64, post=None, gate=None, gs=0, rows=0, res=B, rt=64, h=C, ht=64, w=D, M=4, K=64, eps=1e-6, off=0.0, sc=1.0,
             rs=1.0, dtype=0, out=1, t=None, y=E, ys=None)
    f = caller(lib.sgq_norm, d)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(M=-1), dict(K=0), dict(K=60), dict(K=32776, xt=32776, rt=32776, ht=32776), dict(eps=-1.0), dict(eps=nan),
                dict(off=inf), dict(sc=nan), dict(rs=inf), dict(dtype=2), dict(xt=56), dict(xt=68), dict(rt=8), dict(ht=8),
                dict(out=-1), dict(out=5), dict(out=9), dict(out=64), dict(out=2 | 16 | 32, ys=F), dict(out=2 | 8, ys=F),
                dict(out=3, K=40, ys=F), dict(out=3, ys=F, t=G), dict(out=1, t=G), dict(res=None), dict(h=None),
                dict(res=None, h=None, post=F), dict(res=None, h=None, gate=F, gs=64, rows=4), dict(res=None, h=None, out=0),
                dict(gate=F, gs=64, rows=0), dict(gate=F, gs=8, rows=1), dict(h=A, ht=128), dict(h=B, ht=128), dict(x=None),
                dict(w=None), dict(y=None), dict(out=2), dict(out=4)):
        assert f(**bad) == INV, bad
    for bad in (dict(x=A + 8), dict(res=B + 8), dict(h=C + 2), dict(w=D + 4), dict(y=E + 8), dict(post=F + 8),
                dict(gate=F + 2, gs=64, rows=1), dict(out=2, ys=F + 8), dict(out=4, ys=F, t=G + 1)):
        assert f(**bad) == MIS, bad
    assert f(M=0, x=None, res=None, w=None, y=None) == OK
    assert f(M=0, x=None, res=None, h=None, w=None, y=None) == OK


# ---------------------------------------------------------------- scales' layout

@pytest.mark.parametrize("rows,groups", [(1, 1), (3, 5), (128, 4), (129, 9), (300, 64)])
def test_tiles_are_the_definition(rows, groups):
    s = np.random.default_rng(rows).integers(0, 255, (rows, groups), dtype=np.uint8)
    tiles = sgq.fp4_scales_to_tiles(torch.from_numpy(s))
    assert tiles.shape == (-(-rows // 128), -(-groups // 4), 512)
    assert np.array_equal(tiles.numpy(), ref.to_tiles(s))
    assert np.array_equal(sgq.fp4_scales_from_tiles(tiles, rows, groups).numpy(), s)


def test_tiles_refuse():
    for bad in (torch.zeros(4, dtype=torch.uint8), torch.zeros(4, 4)):
        with pytest.raises(ValueError):
            sgq.fp4_scales_to_tiles(bad)
    with pytest.raises(ValueError):
        sgq.fp4_scales_from_tiles(torch.zeros(1, 2, 512, dtype=torch.uint8), 129, 8)


def test_tensor_scale():
    x = torch.tensor([[1.0, -13.44], [0.0, 2.0]]).bfloat16()
    assert sgq.fp4_tensor_scale(x).item() == pytest.approx(float(x.abs().max()) / 2688, rel=2 ** -23)
    assert sgq.fp4_tensor_scale(torch.zeros(2, 32)).item() == 1.0
    assert sgq.fp4_tensor_scale(torch.full((1,), 1e-41, dtype=torch.float32)).item() >= torch.finfo(torch.float32).tiny


# ---------------------------------------------------------------- what the helpers refuse before a launch

class Recorder:
    """Stands in for the library: records the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def launches(monkeypatch):
    """CPU tensors stand in for a GPU's; a call that reaches the library is recorded instead."""
    r = Recorder()
    monkeypatch.setattr(binding, "_lib", r)
    for m in (fp4, norms):
        monkeypatch.setattr(m, "_current", lambda s: (-1, 0))
        monkeypatch.setattr(m, "_device", lambda *a: None)
    return r.calls


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def refused(f, *a, **k):
    with pytest.raises(ValueError):
        f(*a, **k)


def test_quant_helper_refuses(launches):
    x, t = bf(4, 64), torch.ones(1)
    for args, kw in (((bf(64), "nvfp4"), {}), ((x.float(), "nvfp4"), {}), ((x, "fp4"), {}), ((x, None), {}), ((x, ["nvfp4"]), {}),
                     ((bf(4, 48), "mxfp4"), {}), ((bf(4, 0), "mxfp4"), {}), ((bf(64, 4).t(), "mxfp4"), {}),
                     ((bf(4, 96), "nvfp4"), dict(silu_mul=True)), ((bf(4, 65), "nvfp4"), dict(silu_mul=True)),
                     ((x, "mxfp4"), dict(tensor_scale=t)), ((x, "nvfp4"), dict(tensor_scale=torch.ones(2))),
                     ((x, "nvfp4"), dict(tensor_scale=t.double())), ((x, "nvfp4"), dict(tensor_scale=torch.ones(1, requires_grad=True))),
                     ((x.clone().requires_grad_(), "nvfp4"), {}), ((x, "nvfp4"), dict(xq=u8(4, 64))), ((x, "nvfp4"), dict(xs=u8(1, 2, 512))),
                     ((x, "nvfp4"), dict(xq=bf(4, 32)))):
        refused(sgq.quant_fp4, *args, **kw)
    assert not launches
    with torch.no_grad():
        sgq.quant_fp4(x.clone().requires_grad_(), "nvfp4", tensor_scale=t)
    q, s = sgq.quant_fp4(bf(130, 160)[:, :96], "mxfp4", xq=u8(130, 48))
    assert q.shape == (130, 48) and s.shape == (2, 1, 512) and launches[-1][1][3] == 160 and len(launches) == 2
    sgq.quant_fp4(bf(2, 128), "nvfp4", silu_mul=True)
    assert launches[-1][1][2:4] == (64, 128)
    sgq.quant_fp4(bf(64)[None].expand(1, 64), "nvfp4")
    assert launches[-1][1][1:4] == (1, 64, 64)


def test_packed_helpers_refuse(launches):
    xq, xs, wq, ws, t = u8(4, 32), u8(1, 1, 512), u8(16, 32), u8(1, 1, 512), torch.ones(1)
    g = lambda **k: sgq.fp4_gemm(k.pop("xq", xq), k.pop("xs", xs), k.pop("wq", wq), k.pop("ws", ws), k.pop("fmt", "nvfp4"), **k)  # noqa: E731
    for k in (dict(xq=u8(4)), dict(xq=u8(4, 64)), dict(wq=u8(16, 64)), dict(xs=u8(1, 2, 512)), dict(ws=u8(2, 1, 512)),
              dict(xs=u8(512)), dict(xq=xq.int()), dict(ws=ws.float()), dict(xq=u8(32, 4).t()), dict(fmt="nvfp"), dict(dtype=torch.float32),
              dict(out=bf(4, 8)), dict(out=torch.zeros(4, 16)), dict(out=bf(4, 16), dtype=torch.float16), dict(x_scale=torch.ones(2)),
              dict(w_scale=t.half()), dict(fmt="mxfp4", x_scale=t), dict(x_scale=torch.ones(1, requires_grad=True)),
              dict(out=bf(4, 16).requires_grad_())):
        refused(g, **k)
    d = lambda **k: sgq.dequant_fp4(k.pop("xq", xq), k.pop("xs", xs), k.pop("fmt", "nvfp4"), **k)  # noqa: E731
    for k in (dict(xq=u8(4)), dict(xs=u8(1, 2, 512)), dict(xs=u8(2, 1, 512)), dict(dtype=torch.float32), dict(out=bf(4, 32)),
              dict(fmt="mxfp4", tensor_scale=t), dict(fmt="e2m1"), dict(xq=xq.int())):
        refused(d, **k)
    assert not launches
    out = torch.zeros(4, 16, dtype=torch.float16)
    assert g(out=out, x_scale=t) is out and launches[-1][1][-2] == binding.SGQ_FP16
    assert g().dtype == torch.bfloat16 and d(dtype=torch.float16).shape == (4, 64) and len(launches) == 3


def test_norm_helpers_refuse(launches):
    x, w, r, t = bf(4, 128), bf(128), bf(4, 128), torch.ones(1)
    n = lambda **k: sgq.rms_norm(k.pop("x", x), k.pop("w", w), **k)  # noqa: E731
    for k in (dict(x=bf(128)), dict(x=x.float()), dict(w=w.half()), dict(w=bf(64)), dict(w=bf(1, 128)), dict(x=bf(128, 4).t()),
              dict(w=bf(256)[::2]), dict(x=x.clone().requires_grad_()), dict(w=w.clone().requires_grad_()), dict(quant="int8"),
              dict(quant="fp8", group=64), dict(x=bf(4, 96), w=bf(96), quant="fp8"), dict(quant="fp8", tensor_scale=t),
              dict(quant="fp8_ue8m0", ue8m0=True), dict(quant="nvfp4", ue8m0=True), dict(quant="mxfp4", tensor_scale=t),
              dict(x=bf(4, 48), w=bf(48), quant="nvfp4"), dict(tensor_scale=t), dict(out_scales=t), dict(ue8m0=True), dict(out=bf(4, 64)),
              dict(out=x.half()), dict(quant="fp8", out=bf(4, 128)), dict(quant="fp8", out_scales=u8(4, 1)),
              dict(quant="nvfp4", tensor_scale=torch.ones(1, requires_grad=True))):
        refused(n, **k)
    a = lambda **k: sgq.norm_add(k.pop("x", x), k.pop("r", r), **k)  # noqa: E731
    for k in (dict(r=bf(4, 64)), dict(r=r.half()), dict(r=bf(128, 4).t()), dict(post_weight=bf(64)), dict(post_weight=w.half()),
              dict(weight=bf(64)), dict(gate=bf(3, 128)), dict(gate=bf(4, 64)), dict(gate=bf(0, 128)), dict(gate=bf(128, 4).t()),
              dict(gate=bf(4, 128).half()), dict(h_out=bf(4, 64)), dict(h_out=bf(128, 4).t()), dict(quant="fp8"), dict(out=bf(4, 128)),
              dict(tensor_scale=t), dict(out_scales=t), dict(r=r.clone().requires_grad_()), dict(gate=w.clone().requires_grad_()),
              dict(weight=w.clone().requires_grad_()), dict(post_weight=w.clone().requires_grad_())):
        refused(a, **k)
    assert not launches
    assert n().shape == (4, 128) and isinstance(a(), torch.Tensor)
    h, y = a(weight=w, h_out=r, gate=bf(2, 128))
    assert h is r and y.shape == x.shape
    args = launches[-1][1]
    assert args[4:6] == (128, 2)                        # gate rows, each for two tokens
    h, q, s = a(weight=w, quant="nvfp4", tensor_scale=t, post_weight=w)
    assert q.shape == (4, 64) and s.shape == (1, 2, 512)
    q, s = n(quant="fp8", group=32, ue8m0=True)
    assert s.shape == (4, 4) and s.dtype == torch.float32 and launches[-1][1][18] == binding.SGQ_OUT_FP8 | binding.SGQ_OUT_POW2
    q, s = n(quant="fp8_ue8m0")
    assert s.dtype == torch.uint8 and launches[-1][1][18] == binding.SGQ_OUT_FP8 | binding.SGQ_OUT_GROUP_128 | binding.SGQ_OUT_UE8M0


def test_tensors_elsewhere_are_refused(monkeypatch):
    """CPU tensors, where the current device is a GPU."""
    r = Recorder()
    monkeypatch.setattr(binding, "_lib", r)
    for m in (fp4, norms):
        monkeypatch.setattr(m, "_current", lambda s: (0, 0))
    refused(sgq.quant_fp4, bf(4, 64), "nvfp4")
    refused(sgq.dequant_fp4, u8(4, 32), u8(1, 1, 512), "nvfp4")
    refused(sgq.fp4_gemm, u8(4, 32), u8(1, 1, 512), u8(8, 32), u8(1, 1, 512), "nvfp4")
    refused(sgq.rms_norm, bf(4, 64), bf(64))
    refused(sgq.norm_add, bf(4, 64), bf(4, 64))
    assert not r.calls
