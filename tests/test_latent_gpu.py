"""Latent attention on the GPU against its definition in 64 bits (latent_ref.py)."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
import latent_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def normal(*shape, dtype, seed, std=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


@pytest.fixture(autouse=True)
def status_is_clean():
    yield
    assert sgq.sgq_device_status() == 0


# ---------------------------------------------------------------- rotary

ROTARY = [  # T, H, D, R, offset
    (1, 1, 64, 64, 0), (1, 16, 192, 64, 128), (3, 5, 96, 32, 64), (65, 20, 160, 32, 0), (7, 128, 192, 64, 128),
    (2, 3, 2048, 2048, 0), (2, 9, 2048, 16, 1024), (33, 2, 16, 16, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,D,R,offset", ROTARY)
def test_rotary(T, H, D, R, offset, interleaved, dtype):
    table = sgq.rotary_table(5000, R)
    x = normal(T, H, D, dtype=dtype, seed=1)
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(2))
    pos[0], pos[-1] = 4999, 0
    for inverse in (False, True):
        want, mag = ref.rotate(ref.f64(x), pos.numpy(), ref.f64(table), offset, interleaved, inverse)
        y = sgq.rotary(x, pos.cuda(), table, offset, interleaved, inverse)
        ref.check_rotation(y, want, mag, dtype)
        rest = [c for c in range(D) if not offset <= c < offset + R]
        assert torch.equal(y[..., rest], x[..., rest])
        z = x.clone()
        assert sgq.rotary(z, pos.cuda(), table, offset, interleaved, inverse, out=z) is z
        assert torch.equal(z, y)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_strided_and_empty(interleaved):
    table = sgq.rotary_table(100, 64)
    base = normal(9, 24, 6, 128, dtype=torch.bfloat16, seed=3)
    x = base[:, ::2, 3]                                # strides of neither a token's nor a head's whole rows
    pos = torch.arange(9, device="cuda") * 11
    whole = torch.full((9, 12, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    y = sgq.rotary(x, pos, table, 64, interleaved, out=whole[..., 64:192])
    want, mag = ref.rotate(ref.f64(x), pos.cpu().numpy(), ref.f64(table), 64, interleaved)
    ref.check_rotation(y, want, mag, torch.bfloat16)
    assert (whole[..., :64] == 7).all() and (whole[..., 192:] == 7).all()
    assert sgq.rotary(x[:0], pos[:0], table, 64, interleaved).shape == (0, 12, 128)
    assert sgq.rotary(x[:, :0], pos, table, 64, interleaved).shape == (9, 0, 128)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_inverse_is_the_gradient(interleaved):
    """d <w, rotary(x)> / dx by central differences of the definition, against the inverse rotation of w."""
    table = sgq.rotary_table(300, 32)
    w = normal(4, 3, 32, dtype=torch.float16, seed=5)
    pos = ints([0, 17, 255, 299], torch.int64)
    x, wn, t = ref.f64(normal(4, 3, 32, dtype=torch.float16, seed=6)), ref.f64(w), ref.f64(table)
    grad, h = np.zeros_like(x), 2.0 ** -10
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        f = [(wn * ref.rotate(v, pos.cpu().numpy(), t, 0, interleaved)[0]).sum() for v in (up, down)]
        grad[i] = (f[0] - f[1]) / (2 * h)
    got = sgq.rotary(w, pos, table, 0, interleaved, inverse=True)
    assert np.abs(ref.f64(got) - grad).max() <= 2.0 ** -11 * np.abs(grad).max() + 1e-8


def test_position_outside_the_table_is_reported():
    table = sgq.rotary_table(10, 64)
    x = normal(3, 2, 64, dtype=torch.bfloat16, seed=7)
    y = sgq.rotary(x, ints([1, 10, -1], torch.int64), table)
    assert sgq.sgq_device_status() == 1
    want, mag = ref.rotate(ref.f64(x[:1]), np.array([1]), ref.f64(table), 0, True)
    ref.check_rotation(y[:1], want, mag, torch.bfloat16)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,L,R,page", [(1, 16, 512, 64, 64), (37, 5, 256, 32, 16), (9, 128, 512, 64, 7), (20, 0, 512, 64, 16)])
def test_append(T, H, L, R, page, interleaved, dtype):
    pages = T // page + 5
    table = sgq.rotary_table(1000, R)
    kv = normal(T, L + R, dtype=dtype, seed=1)
    queries = normal(T, max(H, 1), 128 + R, dtype=dtype, seed=2)
    q = queries[:, :H, 128:] if H else None
    pos = torch.randint(0, 1000, (T,), generator=torch.Generator().manual_seed(3))
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(4))[:T]
    if T > 4:
        slots[2], slots[T - 1] = -1, -5
    cache = normal(pages, page + 1, L + R, dtype=dtype, seed=5)[:, :page]      # pages apart by more than a page
    before = cache.clone()
    whole = torch.full((T, max(H, 1), L + R), 3.0, dtype=dtype, device="cuda")
    q_out = whole[:, :H, L:] if H else None
    k_out = torch.empty(T, R, dtype=dtype, device="cuda")
    got = sgq.latent_append(q, kv[:, L:], kv[:, :L], pos.cuda(), slots.cuda(), table, cache, interleaved, q_out, k_out)
    t, p = ref.f64(table), pos.numpy()
    want_k, mag_k = ref.rotate(ref.f64(kv[:, None, L:]), p, t, 0, interleaved)
    ref.check_rotation(k_out, want_k[:, 0], mag_k[:, 0], dtype)
    if H:
        assert got is q_out
        ref.check_rotation(q_out, *ref.rotate(ref.f64(q), p, t, 0, interleaved), dtype)
        assert (whole[..., :L] == 3).all()
        alone = sgq.latent_append(q, kv[:, L:], kv[:, :L], pos.cuda(), slots.cuda(), table, cache, interleaved)
        assert torch.equal(alone, q_out)
    want = before.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // page, s % page, :L] = kv[i, :L]
            want[s // page, s % page, L:] = k_out[i]
    assert torch.equal(cache, want)


def test_append_reports_slots_outside_the_cache():
    table = sgq.rotary_table(10, 64)
    cache = torch.zeros(2, 16, 192, dtype=torch.bfloat16, device="cuda")
    kv = normal(3, 192, dtype=torch.bfloat16, seed=1)
    sgq.latent_append(None, kv[:, 128:], kv[:, :128], ints([1, 2, 3], torch.int64), ints([31, 32, 5], torch.int64),
                      table, cache)
    assert sgq.sgq_device_status() == 1
    assert torch.equal(cache[1, 15, :128], kv[0, :128]) and torch.equal(cache[0, 5, :128], kv[2, :128])
    assert int((cache != 0).any(-1).sum()) == 2


# ---------------------------------------------------------------- absorbed attention

def paged(lens, page, W, dtype, seed, spare=2):
    """A cache whose rows past each request's length, and whose unused pages, hold NaN; a table whose unused entries
    point nowhere."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    cache = torch.full((pages, page, W), float("nan"), dtype=dtype, device="cuda")
    table = torch.full((len(lens), max(max(need), 1)), 2 ** 31 - 1, dtype=torch.int32)
    rows = []
    for b, n in enumerate(lens):
        r = normal(n, W, dtype=dtype, seed=seed * 1000 + b)
        for i in range(need[b]):
            page_no = order.pop()
            table[b, i] = page_no
            part = r[i * page:(i + 1) * page]
            cache[page_no, :part.shape[0]] = part
        rows.append(ref.f64(r))
    return cache, table.cuda(), rows


def check_attention(H, q_lens, kv_lens, L, R, page, dtype, singles=False, std=1.0, cache=None):
    T, W = sum(q_lens), L + R
    cache, table, rows = cache or paged(kv_lens, page, W, dtype, seed=11)
    q = normal(T, H, W, dtype=dtype, seed=12, std=std)
    lse = torch.empty(T, H, dtype=torch.float32, device="cuda")
    scale = 1.0 / math.sqrt(192)
    starts = None if singles else ints(np.concatenate([[0], np.cumsum(q_lens)]).tolist())
    out = sgq.latent_attention(q, cache, table, ints(kv_lens), scale, L, q_starts=starts, lse=lse)
    at = 0
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        visible = np.arange(m)[None] <= (np.arange(n) + m - n)[:, None]
        visible = np.repeat(visible, H, axis=0)
        want = ref.attend(ref.f64(q[at:at + n]).reshape(n * H, W), rows[b], rows[b][:, :L], visible, scale)
        ref.check_rows(out[at:at + n].reshape(n * H, L), lse[at:at + n].reshape(-1), *want, dtype, f"request {b}")
        at += n
    again = sgq.latent_attention(q, cache, table, ints(kv_lens), scale, L, q_starts=starts)
    assert torch.equal(again, out)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 5, 16, 20, 33, 64, 100, 128])
def test_single_tokens(H, dtype):
    lens = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 640, 1023]
    check_attention(H, [1] * len(lens), lens, 512, 64, 16, dtype, singles=True)


@pytest.mark.parametrize("L,R", [(128, 8), (256, 32), (384, 64), (512, 24), (512, 64)])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 256])
def test_widths_and_pages(L, R, page):
    check_attention(16, [1, 1, 1], [300, 77, 129], L, R, page, torch.bfloat16, singles=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 3, 16, 48, 64, 128])
def test_chunks(H, dtype):
    """Chunks at the end of what is cached; one longer than its cache (its first tokens see nothing), one empty."""
    check_attention(H, [1, 5, 0, 37, 140, 9], [400, 5, 33, 37, 300, 4], 512, 64, 32, dtype)


def test_chunk_without_any_row():
    check_attention(16, [3, 2], [0, 2], 512, 64, 16, torch.bfloat16)


@pytest.mark.parametrize("H,lens", [(16, [20000]), (128, [30000]), (8, [1, 40000, 3]), (64, [5000] * 40)])
def test_long_axis_is_split(H, lens):
    check_attention(H, [1] * len(lens), lens, 512, 64, 64, torch.bfloat16, singles=True)


@pytest.mark.parametrize("H", [65, 130, 200, 257, 300])
def test_more_heads_than_a_block(H):
    """Two, three and four head blocks side by side, and more of them one after the other."""
    check_attention(H, [1] * 5, [1000, 3, 0, 129, 2500], 512, 64, 32, torch.bfloat16, singles=True)
    check_attention(H, [3, 1, 40], [300, 2, 45], 256, 32, 16, torch.float16)


def test_tables_without_pages():
    cache = torch.full((2, 16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = normal(3, 16, 576, dtype=torch.bfloat16, seed=1)
    lse = torch.empty(3, 16, device="cuda")
    out = sgq.latent_attention(q, cache, torch.empty(3, 0, dtype=torch.int32, device="cuda"), ints([0, 0, 0]), 0.1, 512, lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_many_requests():
    lens = [(i * 37) % 300 for i in range(700)]
    check_attention(4, [1] * 700, lens, 128, 16, 16, torch.bfloat16, singles=True)


@pytest.mark.parametrize("std", [0.0, 8.0, 40.0])
def test_flat_and_peaked_scores(std):
    """Equal weights, and weights that one key carries: scores spread over hundreds, rising and falling along the axis."""
    check_attention(16, [1, 4], [700, 500], 512, 64, 16, torch.float16, std=std)


@pytest.mark.parametrize("rising", [True, False])
def test_running_maximum_moves(rising):
    """Keys whose scores grow (or shrink) from one tile to the next, so that the sums are rescaled many times."""
    L, R, m, page, H = 512, 64, 2000, 16, 7
    cache, table, _ = paged([m], page, L + R, torch.bfloat16, seed=3)
    step = torch.arange(m, device="cuda", dtype=torch.float32) / m
    rows = (normal(m, L + R, dtype=torch.float32, seed=4) * 0.1 + (step if rising else 1 - step)[:, None]).bfloat16()
    for i in range(m // page):
        cache[table[0, i].long()] = rows[i * page:(i + 1) * page]
    q = (torch.ones(1, H, L + R, device="cuda") * torch.arange(1, H + 1, device="cuda")[:, None]).bfloat16()
    lse = torch.empty(1, H, device="cuda")
    out = sgq.latent_attention(q, cache, table, ints([m]), 0.05, L, lse=lse)
    r = ref.f64(rows)
    want = ref.attend(ref.f64(q[0]), r, r[:, :L], np.ones((H, m), dtype=bool), 0.05)
    ref.check_rows(out[0], lse[0], *want, torch.bfloat16)


def test_offsets_past_32_bits():
    """Pages that lie more than 2^32 bytes apart."""
    L, R, page, H = 512, 64, 16, 16
    W = L + R
    far = (3 << 30) // page // 2 * page // 8 * 8      # elements between pages: 3 GB
    flat = torch.empty(far * 2 + page * W, dtype=torch.bfloat16, device="cuda")
    cache = flat.as_strided((3, page, W), (far, W, 1))
    rows = normal(40, W, dtype=torch.bfloat16, seed=8)
    for i, p in enumerate((2, 0, 1)):
        cache[p] = float("nan")
        part = rows[i * page:(i + 1) * page]
        cache[p, :part.shape[0]] = part
    table = ints([[2, 0, 1]])
    check_attention(H, [1], [40], L, R, page, torch.bfloat16, singles=True, cache=(cache, table, [ref.f64(rows)]))
    check_attention(H, [8], [40], L, R, page, torch.bfloat16, cache=(cache, table, [ref.f64(rows)]))
    t = sgq.rotary_table(8, R)
    kv = normal(1, W, dtype=torch.bfloat16, seed=9)
    sgq.latent_append(None, kv[:, L:], kv[:, :L], ints([0], torch.int64), ints([2 * page + 3], torch.int64), t, cache)
    assert torch.equal(cache[2, 3], kv[0])


def test_strided_queries_and_cache():
    L, R, page, H = 256, 32, 16, 12
    W = L + R
    cache, table, rows = paged([90, 33], page, W, torch.float16, seed=21)
    wide = torch.full((cache.shape[0], page + 2, W + 8), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, :page, :W] = cache
    q = normal(2, H, W + 24, dtype=torch.float16, seed=22)[..., 8:8 + W]
    a = sgq.latent_attention(q, wide[:, :page, :W], table, ints([90, 33]), 0.1, L)
    b = sgq.latent_attention(q.contiguous(), cache, table, ints([90, 33]), 0.1, L)
    assert torch.equal(a, b)
    for i in range(2):
        want = ref.attend(ref.f64(q[i]), rows[i], rows[i][:, :L], np.ones((H, len(rows[i])), dtype=bool), 0.1)
        ref.check_rows(a[i], None, *want, torch.float16)


def test_cache_of_several_layers_side_by_side():
    L, R, page, H = 512, 64, 32, 16
    W = L + R
    lens = [700, 33, 0, 257]
    cache, table, rows = paged(lens, page, W, torch.bfloat16, seed=23)
    layers = torch.full((cache.shape[0], page, 3, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    layers[:, :, 1] = cache
    q = normal(4, H, W, dtype=torch.bfloat16, seed=24)
    a = sgq.latent_attention(q, layers[:, :, 1], table, ints(lens), 0.1, L)
    b = sgq.latent_attention(q, cache, table, ints(lens), 0.1, L)
    assert torch.equal(a, b)


def test_page_and_length_outside_are_reported():
    cache, table, _ = paged([40, 20], 16, 192, torch.bfloat16, seed=1)
    q = normal(2, 4, 192, dtype=torch.bfloat16, seed=2)
    good = sgq.latent_attention(q, cache, table, ints([40, 20]), 0.1, 128)
    assert sgq.sgq_device_status() == 0
    bad = table.clone()
    bad[0, 1] = -3
    out = sgq.latent_attention(q, cache, bad, ints([40, 20]), 0.1, 128)
    assert sgq.sgq_device_status() == 1 and torch.equal(out[1], good[1])
    out = sgq.latent_attention(q, cache, table, ints([-1, 20]), 0.1, 128)
    assert sgq.sgq_device_status() == 1 and torch.equal(out[1], good[1])
    sgq.latent_attention(q, cache, table.clamp(max=3), ints([40, 2000]), 0.1, 128)
    assert sgq.sgq_device_status() == 1


@pytest.mark.parametrize("starts", [[0, 1, 2], [1, 2, 3], [0, 3, 2], [0, 1, 4], [0, -1, 3]])
def test_starts_that_do_not_fit_are_reported(starts):
    cache, table, _ = paged([40, 20], 16, 192, torch.bfloat16, seed=1)
    q = normal(3, 4, 192, dtype=torch.bfloat16, seed=2)
    sgq.latent_attention(q, cache, table, ints([40, 20]), 0.1, 128, q_starts=ints(starts))
    assert sgq.sgq_device_status() == 1
    kv = normal(3, 4, 256, dtype=torch.bfloat16, seed=3)
    kr = normal(3, 64, dtype=torch.bfloat16, seed=4)
    q = normal(3, 4, 192, dtype=torch.bfloat16, seed=5)
    for a, b in ((starts, [0, 1, 3]), ([0, 1, 3], starts)):
        sgq.latent_prefill(q, kv[..., :128], kr, kv[..., 128:], ints(a), ints(b), 0.1)
        assert sgq.sgq_device_status() == 1


def test_workspace_given_and_too_small():
    cache, table, _ = paged([1000, 20], 16, 576, torch.bfloat16, seed=1)
    q, lens = normal(2, 16, 576, dtype=torch.bfloat16, seed=2), ints([1000, 20])
    want = sgq.latent_attention(q, cache, table, lens, 0.1, 512)
    n = sgq.sgq_latent_attention_workspace(2, 16, 512)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # what it holds before does not matter
    for _ in range(2):
        assert torch.equal(sgq.latent_attention(q, cache, table, lens, 0.1, 512, workspace=ws), want)
    with pytest.raises(sgq.SgqError) as e:
        sgq.latent_attention(q, cache, table, lens, 0.1, 512, workspace=ws[:n - 16])
    assert e.value.status == 1


def test_another_stream_and_graph():
    cache, table, _ = paged([1000, 20], 16, 576, torch.bfloat16, seed=1)
    q, lens = normal(2, 16, 576, dtype=torch.bfloat16, seed=2), ints([1000, 20])
    want = sgq.latent_attention(q, cache, table, lens, 0.1, 512)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = sgq.latent_attention(q, cache, table, lens, 0.1, 512, stream=stream)
        s.synchronize()
        assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sgq.latent_attention(q, cache, table, lens, 0.1, 512)
    lens.copy_(ints([517, 300 % 32]))
    want = sgq.latent_attention(q, cache, table, lens, 0.1, 512)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------- expanded attention

def check_prefill(H, q_lens, kv_lens, N, R, dtype, causal=True, std=1.0, poison=()):
    T, S = sum(q_lens), sum(kv_lens)
    q = normal(T, H, N + R, dtype=dtype, seed=31, std=std)
    up = normal(S, H, 2 * N, dtype=dtype, seed=32)
    k, v, k_rot = up[..., :N], up[..., N:], normal(S, 512 + R, dtype=dtype, seed=33)[:, 512:]
    starts = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    kv_starts = np.concatenate([[0], np.cumsum(kv_lens)]).tolist()
    for b in poison:
        up[kv_starts[b]:kv_starts[b + 1]] = float("nan")
    lse = torch.empty(T, H, dtype=torch.float32, device="cuda")
    scale = 1.0 / math.sqrt(N + R)
    out = sgq.latent_prefill(q, k, k_rot, v, ints(starts), ints(kv_starts), scale, causal=causal, lse=lse)
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        if b in poison:
            continue
        visible = np.arange(m)[None] <= (np.arange(n) + m - n)[:, None] if causal else np.ones((n, m), dtype=bool)
        rq, rk = slice(starts[b], starts[b + 1]), slice(kv_starts[b], kv_starts[b + 1])
        for h in range(H):
            keys = np.concatenate([ref.f64(k[rk, h]), ref.f64(k_rot[rk])], axis=1)
            want = ref.attend(ref.f64(q[rq, h]), keys, ref.f64(v[rk, h]), visible.copy(), scale)
            ref.check_rows(out[rq, h], lse[rq, h], *want, dtype, f"request {b}, head {h}")
    again = sgq.latent_prefill(q, k, k_rot, v, ints(starts), ints(kv_starts), scale, causal=causal)
    assert torch.equal(torch.nan_to_num(again), torch.nan_to_num(out))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,q_lens,kv_lens", [
    (1, [1], [1]), (3, [1, 2, 127, 0, 128, 129], [1, 2, 127, 5, 128, 129]), (2, [255, 256, 257], [255, 256, 257]),
    (2, [1, 5, 300], [200, 128, 513]), (2, [9, 300, 4], [4, 130, 0]), (5, [700], [700]),
])
def test_prefill(H, q_lens, kv_lens, causal, dtype):
    check_prefill(H, q_lens, kv_lens, 128, 64, dtype, causal)


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("R", [8, 24, 32, 64])
def test_prefill_widths(N, R):
    check_prefill(4, [77, 200], [77, 300], N, R, torch.bfloat16)


@pytest.mark.parametrize("std", [0.0, 10.0, 60.0])
def test_prefill_flat_and_peaked(std):
    check_prefill(2, [150, 300], [400, 300], 128, 64, torch.float16, std=std)


def test_prefill_requests_do_not_touch():
    """NaN in one request's keys and values stays in that request's rows."""
    check_prefill(2, [100, 40, 130, 5], [100, 40, 130, 5], 128, 64, torch.bfloat16, poison=(1, 3))


def test_prefill_many_requests():
    lens = [(i * 7) % 23 for i in range(90)]
    check_prefill(2, lens, lens, 64, 32, torch.bfloat16)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_more_items_than_sms(causal):
    """CTAs take over items: pairs of query tiles with one and two tiles, without keys, of many lengths."""
    check_prefill(40, [700, 300, 1, 513, 20], [700, 350, 1, 513, 0], 128, 64, torch.bfloat16, causal)


def test_prefill_long():
    check_prefill(2, [3001], [3001], 128, 64, torch.bfloat16)
    check_prefill(1, [130], [4500], 64, 32, torch.float16, causal=False)


def test_prefill_strides_and_alignment():
    """Heads outside tokens, rows with gaps, an output that is aligned to 16 bytes only."""
    T, H = 300, 3
    q = normal(H, T, 192 + 8, dtype=torch.bfloat16, seed=1).transpose(0, 1)[..., 8:]
    k, v = (normal(H, T, 128, dtype=torch.bfloat16, seed=s).transpose(0, 1) for s in (2, 3))
    kr = normal(T, 96, dtype=torch.bfloat16, seed=4)[:, 16:80]
    starts = ints([0, 100, T])
    want = sgq.latent_prefill(q.contiguous(), k.contiguous(), kr.contiguous(), v.contiguous(), starts, starts, 0.1)
    got = sgq.latent_prefill(q, k, kr, v, starts, starts, 0.1)
    assert torch.equal(got, want)
    flat = torch.full((T * H * 128 + 16,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:8 + T * H * 128].view(T, H, 128)
    assert torch.equal(sgq.latent_prefill(q, k, kr, v, starts, starts, 0.1, out=out), want)
    assert (flat[:8] == 5).all() and (flat[-8:] == 5).all()


def test_prefill_another_stream():
    q = normal(300, 2, 192, dtype=torch.bfloat16, seed=1)
    up, kr = normal(300, 2, 256, dtype=torch.bfloat16, seed=2), normal(300, 64, dtype=torch.bfloat16, seed=3)
    args = (q, up[..., :128], kr, up[..., 128:], ints([0, 300]), ints([0, 300]), 0.1)
    want = sgq.latent_prefill(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sgq.latent_prefill(*args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------- the two forms are one operator

def test_absorbed_equals_expanded():
    """With keys k = U_h c and values v = W_h c, the expanded form on (k, v) is the absorbed form on c with queries
    U_h^T q, its rows times W_h: compared in 64 bits through rounded operands, hence the wide bound."""
    H, N, L, R, n = 4, 128, 256, 32, 150
    c = normal(n, L + R, dtype=torch.float16, seed=1)
    up = normal(H, N, L, dtype=torch.float32, seed=2, std=L ** -0.5)
    down = normal(H, N, L, dtype=torch.float32, seed=3, std=L ** -0.5)
    q = normal(n, H, N + R, dtype=torch.float16, seed=4)
    lat = c[:, :L].float()
    k = torch.einsum("hnl,tl->thn", up, lat).half()
    v = torch.einsum("hnl,tl->thn", down, lat).half()
    expanded = sgq.latent_prefill(q, k, c[:, L:], v, ints([0, n]), ints([0, n]), (N + R) ** -0.5)
    qa = torch.cat([torch.einsum("hnl,thn->thl", up, q[..., :N].float()).half(), q[..., N:]], dim=-1)
    cache = torch.zeros(10, 16, L + R, dtype=torch.float16, device="cuda")
    cache.view(-1, L + R)[:n] = c
    o = sgq.latent_attention(qa, cache, torch.arange(10, dtype=torch.int32, device="cuda")[None], ints([n]),
                             (N + R) ** -0.5, L, q_starts=ints([0, n]))
    absorbed = torch.einsum("hnl,thl->thn", down, o.float())
    # operands and outputs rounded to fp16 on the way: a few 2^-11 of values of order 1, scores of order 3
    assert (absorbed - expanded.float()).abs().max() < 0.02


def test_layer_on_all_of_them():
    """A prompt and tokens through FP8 linears and the four operators: the two forms differ by the quantisation of the
    expanded keys' and values' input (E4M3, 3 significand bits after the point: 2^-4 relative at most an element, some
    3% of a row's norm), which both the projections after it and the attention average."""
    from fp8_block_scaled_sgq_gb300 import latent_example
    assert latent_example.main() < 2 ** -4
