"""Latent attention on the GPU where numbers or calls are at the edge, against its definition in 64 bits (latent_ref.py)."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_sgq_gb300 as sgq
import latent_ref as ref

pytestmark = pytest.mark.gpu


def normal(*shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


@pytest.fixture(autouse=True)
def status_is_clean():
    yield
    assert sgq.sgq_device_status() == 0


# ---------------------------------------------------------------- small weights behind a dominant key, fp16

def check_small(got, lse, want, values):
    """The rows' bound, and what fp16 cannot hold of weights below its normal range: they are rounded to a multiple of
    2^-24 as operands that are 2^9 times what they are to the row's largest one, i.e. each is off by 2^-34 of it at
    most, which moves a row by 2^-34 sum_j |v_j|."""
    out, want_lse, mag, e = want
    u = ref.UNIT[torch.float16]
    tol = u * np.abs(out) + (u + 2 * e[:, None] + 2.0 ** -20) * mag + 2.0 ** -25 + 2.0 ** -34 * np.abs(values).sum(axis=0)
    err = np.abs(ref.f64(got) - out)
    assert (err <= tol).all(), f"{(err / tol).max()} times the bound"
    assert (np.abs(ref.f64(lse) - want_lse) <= e + 2.0 ** -18 + 2.0 ** -21 * np.abs(want_lse)).all()


def sink_rows(m, width, depth, at, seed):
    """Values of mean 1/2, and in their first rotated element scores (in powers of two) `depth` or so below row `at`'s,
    whose values are 0."""
    rows = normal(m, width, dtype=torch.float16, seed=seed, mean=0.5)
    rows[:, -64:] = 0
    rows[:, -64] = normal(m, dtype=torch.float16, seed=seed + 1, std=0.25)
    rows[at] = 0
    rows[at, -64] = depth
    return rows


@pytest.mark.parametrize("at", [0, 9000, 19999])
@pytest.mark.parametrize("depth", [12.0, 22.0, 26.0, 31.0])
def test_absorbed_small_weights(depth, at):
    """Many requests that share their pages, so that no row's keys are cut into parts."""
    m, L, page, B = 20000, 128, 32, 304
    rows = sink_rows(m, L + 64, depth, at, seed=41)
    q = torch.zeros(B, 3, L + 64, dtype=torch.float16, device="cuda")
    q[..., L] = 1
    table = torch.arange(m // page, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    lse = torch.empty(B, 3, device="cuda")
    out = sgq.latent_attention(q, rows.view(-1, page, L + 64), table, ints([m] * B), math.log(2.0), L, lse=lse)
    assert torch.equal(out, out[:1, :1].expand_as(out)) and torch.equal(lse, lse[:1, :1].expand_as(lse))
    r = ref.f64(rows)
    want = ref.attend(ref.f64(q[0, :1]), r, r[:, :L], np.ones((1, m), dtype=bool), math.log(2.0))
    check_small(out[0, :1], lse[0, :1], want, r[:, :L])


@pytest.mark.parametrize("at", [0, 9000, 19999])
@pytest.mark.parametrize("depth", [12.0, 22.0, 26.0, 31.0])
def test_expanded_small_weights(depth, at):
    m, N, n = 20000, 64, 130
    rows = sink_rows(m, N + 64, depth, at, seed=43)
    k = torch.zeros(m, 1, N, dtype=torch.float16, device="cuda")
    q = torch.zeros(n, 1, N + 64, dtype=torch.float16, device="cuda")
    q[..., N] = 1
    lse = torch.empty(n, 1, device="cuda")
    out = sgq.latent_prefill(q, k, rows[:, N:], rows[:, None, :N], ints([0, n]), ints([0, m]), math.log(2.0), causal=False,
                             lse=lse)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    r = ref.f64(rows)
    want = ref.attend(ref.f64(q[0, :, N:]), r[:, N:], r[:, :N], np.ones((1, m), dtype=bool), math.log(2.0))
    check_small(out[0], lse[0], want, r[:, :N])


@pytest.mark.parametrize("step", [0.9, 3.9, 7.9, 12.0])
def test_scores_that_rise_from_tile_to_tile(step):
    """By less and by more than a reference follows at once: weights stay finite in fp16."""
    m, L, page = 2000, 128, 16
    rows = normal(m, L + 64, dtype=torch.float16, seed=45)
    rows[:, L:] = 0
    rows[:, L] = (torch.arange(m, device="cuda") // 128 * step).half()
    q = torch.zeros(1, 5, L + 64, dtype=torch.float16, device="cuda")
    q[..., L] = 1
    lse = torch.empty(1, 5, device="cuda")
    out = sgq.latent_attention(q, rows.view(-1, page, L + 64), torch.arange(m // page, dtype=torch.int32, device="cuda")[None],
                               ints([m]), math.log(2.0), L, lse=lse)
    r, seen = ref.f64(rows), np.ones((5, m), dtype=bool)
    ref.check_rows(out[0], lse[0], *ref.attend(ref.f64(q[0]), r, r[:, :L], seen, math.log(2.0)), torch.float16)
    k = torch.zeros(m, 1, L, dtype=torch.float16, device="cuda")
    lse = torch.empty(5, 1, device="cuda")
    out = sgq.latent_prefill(q[0, :, None], k, rows[:, L:], rows[:, None, :L], ints([0, 5]), ints([0, m]), math.log(2.0),
                             causal=False, lse=lse)
    ref.check_rows(out[:, 0], lse[:, 0], *ref.attend(ref.f64(q[0, :, L:]), r[:, L:], r[:, :L], seen, math.log(2.0)), torch.float16)


# ---------------------------------------------------------------- rows whose scores hold NaN

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens", [[300, 0, 5], [70000, 0, 5], [3000, 0, 129] * 30])
def test_nan_queries_are_not_empty_rows(lens, dtype):
    """A query of NaN gives NaN and a NaN logarithm (an item's own row, and one that is joined from few and from many
    parts); without a row to see it is empty like any other.  Its neighbours are what they are without it."""
    L, page, H, B = 128, 64, 5, len(lens)
    width = -(-max(lens) // page)
    cache = normal(width, page, L + 64, dtype=dtype, seed=51)
    table = torch.arange(width, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    q = normal(B, H, L + 64, dtype=dtype, seed=52)
    bad = q.clone()
    bad[:, 1] = float("nan")
    bad[:, 3, 7] = float("nan")
    lse, bad_lse = (torch.empty(B, H, device="cuda") for _ in range(2))
    want = sgq.latent_attention(q, cache, table, ints(lens), 0.1, L, lse=lse)
    got = sgq.latent_attention(bad, cache, table, ints(lens), 0.1, L, lse=bad_lse)
    some = torch.tensor(lens, device="cuda") > 0
    for h in range(H):
        if h in (1, 3):
            assert got[some, h].isnan().all() and bad_lse[some, h].isnan().all()
            assert (got[~some, h] == 0).all() and bad_lse[~some, h].isneginf().all()
        else:
            assert torch.equal(got[:, h], want[:, h]) and torch.equal(bad_lse[:, h], lse[:, h])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_queries_are_not_empty_rows_expanded(dtype):
    T, H, starts, kv_starts = 300, 2, [0, 200, 300], [0, 150, 400]
    up, kr = normal(400, H, 256, dtype=dtype, seed=53), normal(400, 64, dtype=dtype, seed=54)
    q = normal(T, H, 192, dtype=dtype, seed=55)
    bad = q.clone()
    rows = [3, 49, 50, 170, 299]        # (of the first request, rows up to 49 see nothing)
    bad[rows] = float("nan")
    lse, bad_lse = (torch.empty(T, H, device="cuda") for _ in range(2))
    args = (up[..., :128], kr, up[..., 128:], ints(starts), ints(kv_starts), 0.1)
    want = sgq.latent_prefill(q, *args, lse=lse)
    got = sgq.latent_prefill(bad, *args, lse=bad_lse)
    assert got[rows[2:]].isnan().all() and bad_lse[rows[2:]].isnan().all()
    assert (got[rows[:2]] == 0).all() and bad_lse[rows[:2]].isneginf().all()
    rest = [t for t in range(T) if t not in rows]
    assert torch.equal(got[rest], want[rest]) and torch.equal(bad_lse[rest], lse[rest])


# ---------------------------------------------------------------- streams

def test_outputs_belong_to_the_calls_stream(monkeypatch):
    """What a helper allocates comes from the memory of the stream it launches on, the default stream's handle (0)
    included: the handle of a user's current_stream()."""
    kv, pos = normal(2, 192, dtype=torch.bfloat16, seed=1), ints([0, 1], torch.int64)
    table, cache = sgq.rotary_table(4, 64), torch.zeros(2, 16, 192, dtype=torch.bfloat16, device="cuda")
    q, pages, lens = normal(2, 3, 192, dtype=torch.bfloat16, seed=2), ints([[0], [1]]), ints([1, 1])
    up, starts = normal(2, 3, 256, dtype=torch.bfloat16, seed=3), ints([0, 2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    empty, seen = torch.empty, []
    monkeypatch.setattr(torch, "empty", lambda *a, **k: seen.append(torch.cuda.current_stream().cuda_stream) or empty(*a, **k))
    for stream, handle in ((None, 0), (0, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream),
                           (side.cuda_stream, side.cuda_stream)):
        for call in (lambda: sgq.rotary(q, pos, table, 128, stream=stream),
                     lambda: sgq.latent_append(q[..., 128:], kv[:, 128:], kv[:, :128], pos, pos, table, cache, stream=stream),
                     lambda: sgq.latent_attention(q, cache, pages, lens, 0.1, 128, stream=stream),
                     lambda: sgq.latent_prefill(q, up[..., :128], kv[:, 128:], up[..., 128:], starts, starts, 0.1, stream=stream)):
            seen.clear()
            call()
            assert seen and all(s == handle for s in seen), (stream, seen)
        torch.cuda.synchronize()


# ---------------------------------------------------------------- rotation by a scaled table

@pytest.mark.parametrize("interleaved", [True, False])
def test_inverse_is_the_transpose_of_a_scaled_table(interleaved):
    """With an attention factor f the inverse stays the gradient (<w, rotary(x)> = <rotary(w, inverse), x>), and both
    together are f^2 x.  fp16: each of the two rounds once, 2^-11 of what is of order |x| f and |x| f^2."""
    table = sgq.rotary_table(300, 32, factor=4.0, original_max=100, attention_factor=1.5)
    pos = ints([0, 17, 255, 299], torch.int64)
    x, w = (normal(4, 3, 32, dtype=torch.float16, seed=s) for s in (61, 62))
    p, t = pos.cpu().numpy(), ref.f64(table)
    back = sgq.rotary(w, pos, table, 0, interleaved, inverse=True)
    ref.check_rotation(back, *ref.rotate(ref.f64(w), p, t, 0, interleaved, True), torch.float16)
    forth = ref.rotate(ref.f64(x), p, t, 0, interleaved)[0]
    transposed = ref.rotate(ref.f64(w), p, t, 0, interleaved, True)[0]
    assert abs((ref.f64(w) * forth).sum() - (transposed * ref.f64(x)).sum()) < 1e-9
    both = sgq.rotary(sgq.rotary(x, pos, table, 0, interleaved), pos, table, 0, interleaved, inverse=True)
    size = np.abs(ref.f64(x)).max() * 1.5 ** 2 * 2 ** 0.5
    assert np.abs(ref.f64(both) - 2.25 * ref.f64(x)).max() <= 2 * 2.0 ** -11 * size * 2 ** 0.5


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("L,H,B,m", [(512, 16, 1, 128 * 400), (128, 16, 3, 128 * 300), (512, 20, 200, 640), (512, 128, 200, 640)])
def test_absorbed_wait_runs_out_and_the_stream_recovers(L, H, B, m):
    """With SGQ_LATENT_TEST_TIMEOUT the first CTA never loads part of its second tile: the kernel returns on its own, the
    status says so once, and the next call on the stream gives what the one before gave (every CTA's run has more than
    one tile: a long request, some, and many short ones, in the three row blocks)."""
    from fp8_block_scaled_sgq_gb300 import binding
    page, R = 64, 64
    cache = normal(m // page, page, L + R, dtype=torch.bfloat16, seed=71)
    table = torch.arange(m // page, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    q, lens = normal(B, H, L + R, dtype=torch.bfloat16, seed=72), ints([m] * B)
    want = sgq.latent_attention(q, cache, table, lens, 0.05, L)
    ws = torch.empty(sgq.sgq_latent_attention_workspace(B, H, L), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    binding.sgq_latent_attention(q, L + R, B, H, cache, m // page, page, page * (L + R), L + R, L, R, table, m // page, B, lens,
                                 None, 0.05, binding.SGQ_BF16 | binding.SGQ_LATENT_TEST_TIMEOUT, out, None, ws, ws.numel())
    assert sgq.sgq_device_status() == binding.SGQ_ERR_TIMEOUT
    assert sgq.sgq_device_status() == binding.SGQ_OK
    for _ in range(2):
        assert torch.equal(sgq.latent_attention(q, cache, table, lens, 0.05, L), want)
    assert sgq.sgq_device_status() == binding.SGQ_OK


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("T,H", [(300, 1), (1000, 3), (2000, 64)])
def test_expanded_wait_runs_out_and_the_stream_recovers(T, H, N):
    """The same for the expanded form: one item a CTA, and items that CTAs take over."""
    from fp8_block_scaled_sgq_gb300 import binding
    R = 64
    up, kr = normal(T, H, 2 * N, dtype=torch.bfloat16, seed=73), normal(T, R, dtype=torch.bfloat16, seed=74)
    q, starts = normal(T, H, N + R, dtype=torch.bfloat16, seed=75), ints([0, T])
    k, v = up[..., :N], up[..., N:]
    want = sgq.latent_prefill(q, k, kr, v, starts, starts, 0.1)
    out = torch.empty_like(want)
    binding.sgq_latent_prefill(q, H * (N + R), N + R, T, k, H * 2 * N, 2 * N, kr, R, v, H * 2 * N, 2 * N, T, H, N, R, starts, starts,
                               1, 0.1, True, binding.SGQ_BF16 | binding.SGQ_LATENT_TEST_TIMEOUT, out, None)
    assert sgq.sgq_device_status() == binding.SGQ_ERR_TIMEOUT
    assert sgq.sgq_device_status() == binding.SGQ_OK
    for _ in range(2):
        assert torch.equal(sgq.latent_prefill(q, k, kr, v, starts, starts, 0.1), want)
    assert sgq.sgq_device_status() == binding.SGQ_OK


# ---------------------------------------------------------------- calls that overlap, and graphs of them

def layer_calls(dtype, seed):
    """Inputs of all operators and a function that calls each once, in an order that the results depend on: the
    attention reads the rows that the append writes."""
    T, H, L, R, page = 3, 16, 512, 64, 32
    table = sgq.rotary_table(64, R)
    lens = ints([2000, 33, 500])
    width = 63
    pages = torch.randperm(3 * width, generator=torch.Generator().manual_seed(seed)).int().view(3, width).cuda()
    cache = normal(3 * width, page, L + R, dtype=dtype, seed=seed)
    kv, q = normal(T, L + R, dtype=dtype, seed=seed + 1), normal(T, H, L + R, dtype=dtype, seed=seed + 2)
    pos = ints([5, 63, 0], torch.int64)
    slots = torch.stack([pages[b, (n - 1) // page].long() * page + (n - 1) % page for b, n in enumerate((2000, 33, 500))])
    x = normal(700, 4, 192, dtype=dtype, seed=seed + 3)
    up, kr, starts = normal(700, 4, 256, dtype=dtype, seed=seed + 4), normal(700, R, dtype=dtype, seed=seed + 5), ints([0, 301, 700])
    xpos = torch.arange(700, device="cuda") % 64

    def run(stream=None):
        q_rot = sgq.latent_append(q[..., L:], kv[:, L:], kv[:, :L], pos, slots, table, cache, stream=stream)
        o = sgq.latent_attention(q, cache, pages, lens, 0.05, L, stream=stream)
        y = sgq.rotary(x, xpos, table, 128, stream=stream)
        p = sgq.latent_prefill(y, up[..., :128], kr, up[..., 128:], starts, starts, 0.05, stream=stream)
        return q_rot, o, y, p
    return run, (q, kv, x, up)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_two_streams_at_once(dtype):
    """Two callers' work in flight together: each gets what it gets alone, whatever memory the allocator hands out."""
    (a, _), (b, _) = layer_calls(dtype, 100), layer_calls(dtype, 200)
    want = [a(), b()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, run in enumerate((a, b)):
            got[i].append(run(streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outputs in got[i]:
            assert all(torch.equal(g, w) for g, w in zip(outputs, want[i]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_graph_of_all_operators(dtype):
    """A captured step, replayed on new inputs."""
    run, inputs = layer_calls(dtype, 300)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for i in range(3):
        for j, t in enumerate(inputs):
            t.copy_(normal(*t.shape, dtype=dtype, seed=400 + 10 * i + j))
        want = run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
