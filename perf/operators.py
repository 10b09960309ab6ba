"""Latent attention and the steps around it: the cases that are measured, their plain forms and their definition.

Four operators of one attention layer whose keys and values are one shared latent vector a token:

* ``rotary``    rotates part of every head by its token's position (or back again);
* ``append``    rotates the positional parts of queries and keys and writes [latent | key part] rows into a paged cache;
* ``attention`` the absorbed form: every head of every new token against the rows of a paged latent cache;
* ``prefill``   the expanded form: ragged prompts with their own keys and values for each head, causal.

Head counts and widths are those of the projections this repository is tuned for: 24576 = 128 heads x (128 + 64) columns
out of a 1536-wide input, 2048 = 16 heads x 128 into the output projection, prompts of 4096 tokens.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence being generated: every call waits for this one, so latency is all that counts
        {"name": "rotary_one_token", "op": "rotary", "tokens": 1, "heads": 16, "width": 192, "rot": 64, "offset": 128,
         "interleaved": True, "inverse": False, "max_pos": 32768, "dtype": "bf16"},
        # a prompt's queries rotated back (the gradient's direction), all heads, the other layout and type
        {"name": "rotary_prompt_inverse", "op": "rotary", "tokens": 4096, "heads": 128, "width": 192, "rot": 64,
         "offset": 128, "interleaved": False, "inverse": True, "max_pos": 131072, "dtype": "fp16"},
        # one decode step of a batch of 64 with the heads split over eight GPUs
        {"name": "append_decode", "op": "append", "tokens": 64, "heads": 16, "latent": 512, "rot": 64, "width": 192,
         "page": 64, "pages": 256, "interleaved": True, "padded": 0.0, "max_pos": 32768, "dtype": "bf16"},
        # a packed prompt, odd in length, whose last tokens are padding without a slot
        {"name": "append_prompt", "op": "append", "tokens": 4099, "heads": 128, "latent": 512, "rot": 64, "width": 192,
         "page": 16, "pages": 512, "interleaved": False, "padded": 0.02, "max_pos": 131072, "dtype": "fp16"},
        # one short sequence being generated
        {"name": "attention_one_short", "op": "attention", "batch": 1, "heads": 16, "latent": 512, "rot": 64, "page": 64,
         "q_min": 1, "q_max": 1, "kv_min": 1023, "kv_max": 1023, "empty": 0, "ragged": 0, "dtype": "bf16"},
        # a serving batch with the heads split over eight GPUs, lengths over the whole range, one unused place
        {"name": "attention_batch_16_heads", "op": "attention", "batch": 64, "heads": 16, "latent": 512, "rot": 64,
         "page": 64, "q_min": 1, "q_max": 1, "kv_min": 130, "kv_max": 16384, "empty": 1, "ragged": 1, "dtype": "bf16"},
        # one long document, all heads: the split over the long axis
        {"name": "attention_one_long", "op": "attention", "batch": 1, "heads": 128, "latent": 512, "rot": 64, "page": 16,
         "q_min": 1, "q_max": 1, "kv_min": 131071, "kv_max": 131071, "empty": 0, "ragged": 0, "dtype": "fp16"},
        # a large serving batch, all heads on this GPU
        {"name": "attention_batch_128_heads", "op": "attention", "batch": 128, "heads": 128, "latent": 512, "rot": 64,
         "page": 64, "q_min": 1, "q_max": 1, "kv_min": 1024, "kv_max": 8192, "empty": 0, "ragged": 2, "dtype": "bf16"},
        # chunks of new tokens over what the cache holds of their prompts, beside single tokens
        {"name": "attention_chunks", "op": "attention", "batch": 6, "heads": 128, "latent": 512, "rot": 64, "page": 32,
         "q_min": 1, "q_max": 1024, "kv_min": 300, "kv_max": 8000, "empty": 0, "ragged": 3, "dtype": "bf16"},
        # a few short prompts, one of a single token
        {"name": "prefill_short", "op": "prefill", "batch": 3, "heads": 16, "nope": 128, "rot": 64, "q_min": 1,
         "q_max": 300, "prefix": 0, "ragged": 345, "dtype": "bf16"},
        # one prompt of 4096 tokens, all heads
        {"name": "prefill_4096", "op": "prefill", "batch": 1, "heads": 128, "nope": 128, "rot": 64, "q_min": 4096,
         "q_max": 4096, "prefix": 0, "ragged": 0, "dtype": "bf16"},
        # a ragged batch of prompts that continue expanded prefixes, heads split over eight GPUs
        {"name": "prefill_ragged", "op": "prefill", "batch": 8, "heads": 16, "nope": 128, "rot": 64, "q_min": 100,
         "q_max": 8192, "prefix": 2048, "ragged": 5, "dtype": "fp16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _most(op):
    works = [work(c) for c in listed() if c["op"] == op]
    return max(w["bytes"] for w in works), max(w["flops"] for w in works)


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention", "prefill", "prefill"])
    most_bytes, most_flops = _most(op)
    while True:
        rot = rng.choice([64, 64, 64, 32])
        heads = rng.choice([1, 5, 8, 16, 16, 20, 32, 40, 64, 128])
        case = {"op": op, "heads": heads, "rot": rot, "dtype": rng.choice(["bf16", "fp16"])}
        if op == "rotary":
            offset = rng.choice([0, 128])
            case.update(tokens=_log_int(rng, 1, 16384), offset=offset, width=128 + rot,
                        interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, max_pos=131072)
        elif op == "append":
            case.update(tokens=_log_int(rng, 1, 8191), latent=rng.choice([512, 512, 256]), width=128 + rot,
                        page=rng.choice([16, 32, 64, 128]), interleaved=rng.random() < 0.5,
                        padded=rng.choice([0.0, 0.1]), max_pos=131072)
            case["pages"] = case["tokens"] // case["page"] + rng.randint(1, 64)
        elif op == "attention":
            q_max = rng.choice([1, 1, 1, 5, 700])
            kv_max = _log_int(rng, 1, 131072)
            case.update(batch=_log_int(rng, 1, 256), latent=rng.choice([512, 512, 256]),
                        page=rng.choice([16, 32, 64, 128]), q_min=1, q_max=q_max, kv_min=max(1, kv_max // rng.choice([1, 2, 16])),
                        kv_max=kv_max, empty=0, ragged=rng.randint(0, 10 ** 6))
            case["empty"] = 1 if case["batch"] > 4 and rng.random() < 0.5 else 0
        else:
            q_max = _log_int(rng, 1, 16384)
            case.update(batch=_log_int(rng, 1, 32), nope=rng.choice([128, 128, 64]), q_min=max(1, q_max // 16), q_max=q_max,
                        prefix=rng.choice([0, 0, 500, 2048]), ragged=rng.randint(0, 10 ** 6))
        w = work(case)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return case


def _lengths(case):
    """New tokens and all tokens (with what is cached) of every request: drawn from the case alone."""
    rng = random.Random(case["ragged"])
    q, kv = [], []
    for i in range(case["batch"]):
        n = _log_int(rng, case["q_min"], case["q_max"])
        if case["op"] == "attention":
            have = _log_int(rng, case["kv_min"], case["kv_max"])
            if i < case["empty"]:
                n, have = 1, 0          # a place of a padded batch that holds no request
            else:
                have = max(have, n)
        else:
            have = n + (rng.randint(0, case["prefix"]) if case["prefix"] else 0)
        q.append(n)
        kv.append(have)
    return q, kv


def _pairs(q, kv):
    """Query-key pairs that a causal mask leaves."""
    return sum(n * m - n * (n - 1) // 2 if m >= n else 0 for n, m in zip(q, kv))


def work(case):
    op, heads, rot = case["op"], case["heads"], case["rot"]
    if op == "rotary":
        n = case["tokens"] * heads
        return {"bytes": 4 * n * case["width"] + case["tokens"] * (4 * rot + 8), "flops": 3 * n * rot}
    if op == "append":
        t, row = case["tokens"], case["latent"] + rot
        held = t - int(t * case["padded"])
        return {"bytes": 4 * t * heads * rot + t * (4 * rot + 16) + 4 * held * row, "flops": 3 * rot * (t * heads + held)}
    q, kv = _lengths(case)
    if op == "attention":
        row = case["latent"] + rot
        return {"bytes": 2 * sum(kv) * row + 2 * sum(q) * heads * (row + case["latent"]),
                "flops": 2 * _pairs(q, kv) * heads * (row + case["latent"])}
    width = case["nope"] + rot
    return {"bytes": 2 * heads * (sum(q) * (width + case["nope"]) + sum(kv) * 2 * case["nope"]) + 2 * sum(kv) * rot,
            "flops": 2 * _pairs(q, kv) * heads * (width + case["nope"])}


# ---------------------------------------------------------------- inputs

def _table(max_pos, rot):
    """fp32 [max_pos, rot]: cosines, then sines, of position x 10000^(-2i/rot)."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def _starts(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, heads, rot = DTYPES[case["dtype"]], case["heads"], case["rot"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "rotary":
        t = case["tokens"]
        s["x"] = normal(t, heads, case["width"])
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda")
        s["table"] = _table(case["max_pos"], rot)
    elif case["op"] == "append":
        t, latent = case["tokens"], case["latent"]
        q = normal(t, heads, case["width"])             # rows of the query projection: [plain part | rotated part]
        kv = normal(t, latent + rot)                    # rows of the latent projection: [latent | key part]
        s["q_rot"], s["latent"], s["k_rot"] = q[..., -rot:], kv[:, :latent], kv[:, latent:]
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda")
        slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:t]
        held = t - int(t * case["padded"])
        slots[held:] = -1
        s["slots"], s["held"] = slots, held
        s["table"] = _table(case["max_pos"], rot)
        s["cache"] = normal(case["pages"], case["page"], latent + rot)
    elif case["op"] == "attention":
        q_len, kv_len = _lengths(case)
        latent, page = case["latent"], case["page"]
        need = [-(-n // page) for n in kv_len]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(case["batch"], max(1, max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["cache"] = normal(pages, page, latent + rot)
        # spread so that a few keys carry most of a row's weight, as they do in trained models
        s["q"] = normal(sum(q_len), heads, latent + rot, std=1.2)
        s["page_table"], s["kv_lens"] = table, torch.tensor(kv_len, dtype=torch.int32, device="cuda")
        s["q_starts"] = None if case["q_max"] == 1 else _starts(q_len)
        s["scale"] = 1.0 / math.sqrt(128 + rot)
        s["lengths"] = (q_len, kv_len)
    else:
        q_len, kv_len = _lengths(case)
        nope = case["nope"]
        s["q"] = normal(sum(q_len), heads, nope + rot, std=1.5)
        up = normal(sum(kv_len), heads, 2 * nope)       # the latent vectors' up-projection: [keys | values] of every head
        s["k"], s["v"] = up[..., :nope], up[..., nope:]
        s["k_rot"] = normal(sum(kv_len), 512 + rot)[:, 512:]
        s["q_starts"], s["kv_starts"] = _starts(q_len), _starts(kv_len)
        s["scale"] = 1.0 / math.sqrt(nope + rot)
        s["lengths"] = (q_len, kv_len)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import fp8_block_scaled_sgq_gb300 as sgq

    case = s["case"]
    if case["op"] == "rotary":
        return sgq.rotary(s["x"], s["positions"], s["table"], offset=case["offset"], interleaved=case["interleaved"],
                          inverse=case["inverse"])
    if case["op"] == "append":
        q = sgq.latent_append(s["q_rot"], s["k_rot"], s["latent"], s["positions"], s["slots"], s["table"], s["cache"],
                              interleaved=case["interleaved"])
        return {"q": q, "cache": s["cache"]}
    if case["op"] == "attention":
        return sgq.latent_attention(s["q"], s["cache"], s["page_table"], s["kv_lens"], s["scale"], case["latent"],
                                    q_starts=s["q_starts"])
    return sgq.latent_prefill(s["q"], s["k"], s["k_rot"], s["v"], s["q_starts"], s["kv_starts"], s["scale"])


def _rotate(x, cos, sin, interleaved):
    """x [..., rot] in fp32; cos, sin [..., rot / 2]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rotary":
        rot, off = case["rot"], case["offset"]
        cos, sin = s["table"][s["positions"]].chunk(2, dim=-1)
        if case["inverse"]:
            sin = -sin
        y = s["x"].clone()
        part = s["x"][..., off:off + rot].float()
        y[..., off:off + rot] = _rotate(part, cos[:, None], sin[:, None], case["interleaved"]).to(y.dtype)
        return y
    if case["op"] == "append":
        cos, sin = s["table"][s["positions"]].chunk(2, dim=-1)
        q = _rotate(s["q_rot"].float(), cos[:, None], sin[:, None], case["interleaved"]).to(s["q_rot"].dtype)
        k = _rotate(s["k_rot"].float(), cos, sin, case["interleaved"]).to(s["k_rot"].dtype)
        rows = s["cache"].view(-1, s["cache"].shape[-1])
        held = s["held"]
        rows[s["slots"][:held]] = torch.cat([s["latent"], k], dim=-1)[:held]
        return {"q": q, "cache": s["cache"]}
    if case["op"] == "attention":
        if case["q_max"] == 1:
            return _plain_single(s, case["latent"])
        return _plain_chunks(s, case["latent"])
    return _plain_prefill(s)


def _plain_single(s, latent):
    """One query token a request: all requests at once over rows padded to the longest."""
    q, cache, page = s["q"], s["cache"], s["cache"].shape[1]
    most = s["page_table"].shape[1] * page
    out = torch.empty(q.shape[0], q.shape[1], latent, dtype=q.dtype, device=q.device)
    step = max(1, (1 << 31) // (most * cache.shape[-1]))
    for b in range(0, q.shape[0], step):
        rows = cache[s["page_table"][b:b + step].long()].flatten(1, 2).float()
        lens = s["kv_lens"][b:b + step]
        alive = torch.arange(most, device=q.device) < lens[:, None]
        rows = rows.masked_fill(~alive[..., None], 0.0)
        scores = torch.bmm(q[b:b + step].float(), rows.transpose(1, 2)) * s["scale"]
        scores = scores.masked_fill(~alive[:, None], float("-inf"))
        top = scores.amax(dim=-1, keepdim=True)
        p = torch.exp(scores - torch.where(top.isinf(), 0.0, top))
        o = torch.bmm(p, rows[..., :latent]) / p.sum(dim=-1, keepdim=True).clamp_min(1e-30)
        out[b:b + step] = o.to(q.dtype)
    return out


def _softmax_product(scores, alive, values):
    scores = scores.masked_fill(~alive, float("-inf"))
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(top.isinf(), 0.0, top))
    return torch.matmul(p, values) / p.sum(dim=-1, keepdim=True).clamp_min(1e-30)


def _plain_chunks(s, latent):
    """Requests one after the other, a block of their new tokens at a time."""
    q, cache, page = s["q"], s["cache"], s["cache"].shape[1]
    heads = q.shape[1]
    out = torch.empty(q.shape[0], heads, latent, dtype=q.dtype, device=q.device)
    at = 0
    for i, (n, m) in enumerate(zip(*s["lengths"])):
        if m == 0:
            out[at:at + n] = 0
            at += n
            continue
        rows = cache[s["page_table"][i, :-(-m // page)].long()].flatten(0, 1)[:m].float()
        step = max(1, (1 << 28) // (heads * m))
        for t in range(0, n, step):
            k = min(step, n - t)
            part = q[at + t:at + t + k].float()
            alive = torch.arange(m, device=q.device) <= torch.arange(t, t + k, device=q.device)[:, None] + (m - n)
            scores = torch.matmul(part, rows.T) * s["scale"]
            o = _softmax_product(scores, alive[:, None], rows[:, :latent])
            out[at + t:at + t + k] = o.to(q.dtype)
        at += n
    return out


def _plain_prefill(s):
    """Requests one after the other, a block of heads at a time."""
    q, heads = s["q"], s["q"].shape[1]
    out = torch.empty(q.shape[0], heads, s["v"].shape[-1], dtype=q.dtype, device=q.device)
    at = kv_at = 0
    for n, m in zip(*s["lengths"]):
        alive = torch.arange(m, device=q.device) <= torch.arange(n, device=q.device)[:, None] + (m - n)
        step = max(1, (1 << 29) // (n * m))
        for h in range(0, heads, step):
            qh = q[at:at + n, h:h + step].float().transpose(0, 1)
            kh = s["k"][kv_at:kv_at + m, h:h + step].float()
            kr = s["k_rot"][kv_at:kv_at + m, None].float().expand(-1, kh.shape[1], -1)
            kh = torch.cat([kh, kr], dim=-1).transpose(0, 1)
            vh = s["v"][kv_at:kv_at + m, h:h + step].float().transpose(0, 1)
            scores = torch.bmm(qh, kh.transpose(1, 2)) * s["scale"]
            out[at:at + n, h:h + step] = _softmax_product(scores, alive, vh).transpose(0, 1).to(q.dtype)
        at += n
        kv_at += m
    return out


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotation(s["x"], s, case["offset"], case["interleaved"], case["inverse"])
    if case["op"] == "append":
        q = _exact_rotation(s["q_rot"], s, 0, case["interleaved"], False)
        k = _exact_rotation(s["k_rot"][:, None], s, 0, case["interleaved"], False)[:, 0]
        cache = s["cache"].double()
        page = cache.shape[1]
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                row = cache[slot // page, slot % page]
                row[:case["latent"]] = s["latent"][t].double()
                row[case["latent"]:] = k[t]
        return {"q": q, "cache": cache}
    q_len, kv_len = s["lengths"]
    out, at, kv_at = [], 0, 0
    for i, (n, m) in enumerate(zip(q_len, kv_len)):
        q = s["q"][at:at + n]
        if case["op"] == "attention":
            where = torch.arange(m, device="cuda")
            page = s["cache"].shape[1]
            rows = s["cache"][s["page_table"][i].long()[where // page], where % page].double()
            out.append(_exact_rows(q, lambda h: (rows, rows[:, :case["latent"]]), n, m, s["scale"], case["latent"]))
        else:
            kr = s["k_rot"][kv_at:kv_at + m].double()

            def own_rows(h, lo=kv_at, hi=kv_at + m, kr=kr):
                return torch.cat([s["k"][lo:hi, h].double(), kr], dim=1), s["v"][lo:hi, h].double()

            out.append(_exact_rows(q, own_rows, n, m, s["scale"], case["nope"]))
        at += n
        kv_at += m
    return torch.cat(out)


def _exact_rotation(x, s, offset, interleaved, inverse):
    """Each pair as a complex number, times e^(i angle) (its conjugate for the way back), angle's parts from the table."""
    half = s["table"].shape[1] // 2
    w = s["table"][s["positions"]].double()
    turn = torch.complex(w[:, :half], -w[:, half:] if inverse else w[:, half:])[:, None]
    y = x.double()
    first = offset + torch.arange(half, device="cuda") * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first] = z.real
    y[..., second] = z.imag
    return y


def _exact_rows(q, rows_of, n, m, scale, width):
    """sum_j exp(s_j - log sum_j exp s_j) v_j over the keys j <= m - n + i of new token i, head by head; nothing where there are none."""
    out = torch.zeros(n, q.shape[1], width, dtype=torch.float64, device="cuda")
    if m == 0:
        return out
    last = torch.arange(n, device="cuda") + (m - n)
    for h in range(q.shape[1]):
        k, v = rows_of(h)
        for t in range(0, n, 2048):
            s = (q[t:t + 2048, h].double() @ k.T) * scale
            s[torch.arange(m, device="cuda")[None] > last[t:t + 2048, None]] = -math.inf
            whole = torch.logsumexp(s, dim=1, keepdim=True)
            w = torch.where(torch.isinf(whole), torch.zeros_like(s), torch.exp(s - whole))
            out[t:t + 2048, h] = w @ v
    return out
