"""Latent attention's helpers without a GPU: rotary tables of long contexts."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
from fp8_block_scaled_sgq_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


# ---------------------------------------------------------------- rotary tables of stretched contexts

def table_by_parts(max_pos, rot, base, factor, trained, fast=32.0, slow=1.0):
    """Pair i turns trained base^(-2i/rot) / (2 pi) times over the trained length.  The pairs at which that is `fast` and
    `slow` (rounded outwards, the first one not below 0) bound the blend, linear in i."""
    def pair_at(turns):
        return rot / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)
    lo, hi = max(math.floor(pair_at(fast)), 0), math.ceil(pair_at(slow))
    keep = [0.0 if i >= hi else 1.0 if i <= lo else (hi - i) / (hi - lo) for i in range(rot // 2)]
    freq = [base ** (-2.0 * i / rot) * (k + (1 - k) / factor) for i, k in enumerate(keep)]
    angle = np.arange(max_pos, dtype=np.float64)[:, None] * np.array(freq)
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1), keep


@pytest.mark.parametrize("rot,base,trained", [
    (64, 10000.0, 1000), (64, 10000.0, 4096), (64, 10000.0, 65536), (64, 10000.0, 131072), (32, 10000.0, 1 << 20),
    (128, 500000.0, 8192), (64, 10000.0, 100), (64, 10000.0, 5),
])
def test_table_by_parts_is_the_definition(rot, base, trained):
    """From trained lengths over which every pair turns more often than `slow` (the blend ends past the last pair: 65536,
    131072, 2^20) to one over which none does (5).  Both sides round an angle's 64-bit cosine to fp32 once: 2^-25 of 1,
    and angles up to 2000 in 64 bits differ by less than 2^-40."""
    want, keep = table_by_parts(2000, rot, base, 8.0, trained)
    got = sgq.rotary_table(2000, rot, base=base, factor=8.0, original_max=trained, device="cpu").double().numpy()
    assert np.abs(got - want).max() <= 2.0 ** -25 + 2.0 ** -40
    if trained == 131072:
        assert keep[28] == pytest.approx(0.538, abs=1e-3) and keep[31] == pytest.approx(0.308, abs=1e-3)


# ---------------------------------------------------------------- what the helpers refuse before a launch

@pytest.fixture
def launches(monkeypatch):
    """CPU tensors stand in for a GPU's; a call that reaches the library is recorded instead."""
    calls = []
    monkeypatch.setattr("fp8_block_scaled_sgq_gb300.latent._device", lambda *a: None)
    monkeypatch.setattr("fp8_block_scaled_sgq_gb300.binding._stream", lambda s: 0)
    for name in ("sgq_rotary", "sgq_latent_append", "sgq_latent_attention", "sgq_latent_prefill"):
        monkeypatch.setattr(f"fp8_block_scaled_sgq_gb300.binding.{name}", lambda *a, n=name: calls.append((n, a)))
    return calls


def attention_args():
    q, cache = torch.zeros(2, 16, 192, dtype=torch.bfloat16), torch.zeros(2, 16, 192, dtype=torch.bfloat16)
    pages, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    return q, cache, pages, lens, 0.1, 128


def test_workspace_has_to_be_contiguous(launches):
    """Elements that share memory, or lie apart, are no workspace of numel() elements."""
    sgq.latent_attention(*attention_args(), workspace=torch.empty(1 << 20, dtype=torch.uint8))
    sgq.latent_attention(*attention_args(), workspace=torch.empty(1 << 10, 1 << 8))
    assert [a[-2] for _, a in launches] == [1 << 20, 1 << 20]
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(1 << 20, dtype=torch.uint8)[::2],
                torch.empty(1 << 10, 1 << 8).t()):
        with pytest.raises(ValueError, match="workspace"):
            sgq.latent_attention(*attention_args(), workspace=bad)
    assert len(launches) == 2


class OnDevice:
    is_cuda = True

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """A call's stream, workspace and launch are the current device's."""
    from fp8_block_scaled_sgq_gb300 import latent
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    latent._device(OnDevice(0), None, OnDevice(0))
    with pytest.raises(ValueError, match="different devices"):
        latent._device(OnDevice(0), OnDevice(1))
    with pytest.raises(ValueError, match="current"):
        latent._device(OnDevice(1), None, OnDevice(1))


@pytest.fixture
def sizes_asked_anew():
    """No workspace size of this test is kept for others, and none of theirs for this one."""
    from fp8_block_scaled_sgq_gb300 import latent
    latent._workspace_bytes.cache_clear()
    yield
    latent._workspace_bytes.cache_clear()


def test_workspace_size_is_a_devices(monkeypatch, sizes_asked_anew):
    """Its size goes by the device's number of SMs: one that was asked for on another device is not taken."""
    from fp8_block_scaled_sgq_gb300 import latent
    device = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: device[0])
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda n, *a, **k: 16)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda p: None)
    monkeypatch.setattr(binding, "sgq_latent_attention_workspace", lambda T, H, L: 1000 * (1 + device[0]))
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    monkeypatch.setattr(latent, "_device", lambda x, *a: device[0])
    sizes = []
    monkeypatch.setattr(binding, "sgq_latent_attention", lambda *a: sizes.append(a[-2]))
    for device[0] in (0, 1, 0):
        sgq.latent_attention(*attention_args())
    assert sizes == [1000, 2000, 1000]


# ---------------------------------------------------------------- the C ABI's bounds

def test_products_of_sizes_that_wrap(lib):
    """Token and table counts whose products with heads and pages pass 2^63 (and would wrap to small numbers)."""
    import ctypes
    from test_latent import ATT, INV, caller
    f = caller(lib.sgq_latent_attention, list(ATT), ATT)
    fake = 0x70000
    for bad in (dict(T=1 << 48, H=65535, starts=fake), dict(T=(1 << 62) + 4, starts=fake), dict(T=1 << 31, H=1, starts=fake),
                dict(page=1 << 30, width=1, cr=1 << 40, cp=1 << 40), dict(width=1 << 60), dict(width=1 << 62, page=32, cp=18432), dict(width=1 << 31, page=16)):
        assert f(**bad) == INV, bad
    n = ctypes.c_int64()
    for bad in ((1 << 48, 65535, 512), ((1 << 62) + 4, 16, 512), (1 << 27, 16, 512)):
        assert lib.sgq_latent_attention_workspace(*bad, ctypes.byref(n)) == INV, bad


def test_what_the_library_refuses_is_a_value_error(lib, monkeypatch):
    """Shapes, strides and addresses that only the C ABI looks at: ValueError (and SgqError with its status)."""
    monkeypatch.setattr("fp8_block_scaled_sgq_gb300.latent._device", lambda *a: 0)
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    bf16, ws = torch.bfloat16, torch.empty(1 << 10, dtype=torch.uint8)
    pages, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)

    def attention(page=16, width=192, latent=128, gap=0, skip=0):
        q = torch.zeros(2 * 16 * (width + gap) + 8, dtype=bf16)[skip:skip + 2 * 16 * (width + gap)].view(2, 16, width + gap)
        return lambda: sgq.latent_attention(q[..., :width], torch.zeros(2, page, width, dtype=bf16), pages, lens, 0.1, latent,
                                            workspace=ws)

    def prefill(plain, rot):
        k = torch.zeros(2, 3, plain, dtype=bf16)
        return lambda: sgq.latent_prefill(torch.zeros(2, 3, plain + rot, dtype=bf16), k, torch.zeros(2, rot, dtype=bf16), k,
                                          lens, lens, 0.1)

    def rotate(rot, offset=0, interleaved=True):
        return lambda: sgq.rotary(torch.zeros(2, 3, 64, dtype=bf16), torch.zeros(2, dtype=torch.int64), torch.zeros(4, rot),
                                  offset, interleaved)

    kv, pos = torch.zeros(2, 128 + 64 + 4, dtype=bf16), torch.zeros(2, dtype=torch.int64)
    refused = [(attention(page=24), 1), (attention(width=164, latent=100), 1), (attention(width=200), 1), (attention(gap=4), 1),
               (attention(skip=4), 3), (prefill(96, 64), 1), (prefill(128, 72), 1), (rotate(12), 1), (rotate(24, 0, False), 1),
               (rotate(32, 40), 1),
               (lambda: sgq.latent_append(None, kv[:, 128:192], kv[:, :128], pos, pos, torch.zeros(4, 64),
                                          torch.zeros(2, 16, 192, dtype=bf16)), 1)]
    for call, status in refused:
        with pytest.raises(ValueError) as e:
            call()
        assert isinstance(e.value, sgq.SgqError) and e.value.status == status
    # what is not about arguments stays an SgqError alone
    assert not isinstance(binding.SgqError(binding.SGQ_ERR_CUDA, "call"), ValueError)


def test_inputs_that_require_a_gradient(launches):
    """No operator records one: refused while gradients are recorded, instead of an output that has lost it."""
    bf16 = torch.bfloat16
    pos, table, starts = torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64), torch.zeros(3, dtype=torch.int32)

    def zeros(*shape):
        return torch.zeros(*shape, dtype=bf16)

    def rotary(x):
        sgq.rotary(x, pos, table)

    def append(q, k, latent):
        sgq.latent_append(q, k, latent, pos, pos, table, zeros(2, 16, 192))

    def attention(q, cache):
        sgq.latent_attention(q, cache, *attention_args()[2:], workspace=torch.empty(16))

    def prefill(q, k, k_rot, v):
        sgq.latent_prefill(q, k, k_rot, v, starts, starts, 0.1)

    for call, args in ((rotary, [zeros(2, 3, 64)]), (append, [zeros(2, 3, 64), zeros(2, 64), zeros(2, 128)]),
                       (attention, [zeros(2, 16, 192), zeros(2, 16, 192)]),
                       (prefill, [zeros(2, 3, 192), zeros(2, 3, 128), zeros(2, 64), zeros(2, 3, 128)])):
        for i in range(len(args)):
            graded = [t.requires_grad_() if j == i else t for j, t in enumerate(t.detach() for t in args)]
            with pytest.raises(ValueError, match="gradient"):
                call(*graded)
            assert not launches
            with torch.no_grad():
                call(*graded)
            call(*[t.detach() for t in graded])
            assert len(launches) == 2
            launches.clear()


# ---------------------------------------------------------------- torch's public interface

def test_public_names_of_torch_do(monkeypatch, sizes_asked_anew):
    """The current stream and the workspace's memory, where torch has no names but its public ones."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice", "_cuda_cudaCachingAllocator_raw_alloc",
                 "_cuda_cudaCachingAllocator_raw_delete"):
        monkeypatch.delattr(torch._C, name, raising=False)
    stream = type("Stream", (), {"cuda_stream": 7})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    assert binding._stream(None) == 7 and binding._stream(stream) == 7 and binding._stream(5) == 5
    held, calls = [], []
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda n, device, stream: held.append((n, device, stream)) or 64)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda p: held.remove((512, 0, 7)) if p == 64 else None)
    monkeypatch.setattr("fp8_block_scaled_sgq_gb300.latent._device", lambda *a: 0)
    monkeypatch.setattr(binding, "sgq_latent_attention_workspace", lambda *a: 512)
    monkeypatch.setattr(binding, "sgq_latent_attention", lambda *a: calls.append((list(held), a[-3:])))
    sgq.latent_attention(*attention_args())
    assert calls == [([(512, 0, 7)], (64, 512, 7))] and held == []


# ---------------------------------------------------------------- other devices

STUBS = r"""
// What latent_attn.cu and latent_prefill.cu need of the library's other files, on a device of the given capability.
#include "sgq_internal.h"
namespace sgq {
static DeviceInfo g_device;
sgq_status device_info(DeviceInfo* out) { *out = g_device; return SGQ_OK; }
void note_launch(int) {}
namespace gemm {
sgq_status status_word(uint32_t** out) { *out = nullptr; return SGQ_ERR_CUDA; }
sgq_status get_encoder(TensorMapEncoder* out) { *out = nullptr; return SGQ_ERR_CUDA; }
}
}
extern "C" int attention_on(int major, int minor) {
    sgq::g_device.cc_major = major; sgq::g_device.cc_minor = minor; sgq::g_device.sm_count = 152;
    return sgq::launch_latent_attention(sgq::LatentArgs{}, nullptr);
}
extern "C" int prefill_on(int major, int minor) {
    sgq::g_device.cc_major = major; sgq::g_device.cc_minor = minor; sgq::g_device.sm_count = 152;
    return sgq::launch_latent_prefill(sgq::PrefillArgs{}, nullptr);
}
"""


def test_devices_that_the_library_is_not_built_for(lib, tmp_path):
    """Compiled for 10.3 alone: any other device is SGQ_ERR_UNSUPPORTED, before anything is asked of the driver (where
    the stubs return SGQ_ERR_CUDA)."""
    import ctypes
    import os
    import subprocess
    objects = [os.path.join(build.BUILD, f) for f in ("latent_attn.o", "latent_prefill.o")]
    if not all(map(os.path.exists, objects)):
        build.build(force=True)
    src, so = tmp_path / "stubs.cpp", tmp_path / "stubs.so"
    src.write_text(STUBS)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-I", build.CSRC, "-shared", str(src),
                    *objects, "-o", str(so)], check=True)
    stubs = ctypes.CDLL(str(so))
    for f in (stubs.attention_on, stubs.prefill_on):
        for major, minor in ((10, 0), (10, 1), (9, 0), (12, 0), (11, 3)):
            assert f(major, minor) == binding.SGQ_ERR_UNSUPPORTED, (major, minor)
        assert f(10, 3) == binding.SGQ_ERR_CUDA
