"""A block of linears in 4 bits: the cases that are measured, their plain forms and their definition.

* ``quant``  a 16-bit tensor to 4-bit codes with microscales, and back to the values that these stand for;
* ``gemm``   the product of two tensors in that form;
* ``norm``   the norm before a block, or after it with its gate, its scale and the residual, and the next norm, in 16 bits
  or in FP8 groups;
* ``linear`` a 4-bit linear as it is run: a norm, or silu(gate) * up, written in 4 bits, and the product that reads it.

Formats: "mxfp4", 32 values a scale, a power of two; "nvfp4", 16 values a scale, E4M3, and one fp32 scale a tensor.
Sizes are those of the linears that this repository is tuned for: (N, K) = (7168, 2048), (24576, 1536), (1536, 7168),
(7168, 7168).
"""
import math
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = {"mxfp4": 32, "nvfp4": 16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the activations of one sequence being generated: latency is all that counts
        {"name": "quant_one_token", "op": "quant", "m": 1, "k": 7168, "fmt": "nvfp4", "pad": 0, "dtype": "bf16"},
        # a packed prompt, odd in length, inside wider rows (one part of a joined projection)
        {"name": "quant_prompt_odd", "op": "quant", "m": 4099, "k": 7168, "fmt": "mxfp4", "pad": 576, "dtype": "fp16"},
        # one sequence being generated: the weights' bytes and latency
        {"name": "gemm_one_token", "op": "gemm", "m": 1, "n": 7168, "k": 2048, "fmt": "nvfp4", "dtype": "bf16"},
        # a decode step of a batch of 64 through the widest projection
        {"name": "gemm_batch_64", "op": "gemm", "m": 64, "n": 24576, "k": 1536, "fmt": "mxfp4", "dtype": "bf16"},
        # a short chunk, odd in length, through the narrowest one: few tiles, a long sum
        {"name": "gemm_chunk_odd", "op": "gemm", "m": 301, "n": 1536, "k": 7168, "fmt": "nvfp4", "dtype": "fp16"},
        # a prompt, long sums
        {"name": "gemm_prompt", "op": "gemm", "m": 4096, "n": 7168, "k": 7168, "fmt": "nvfp4", "dtype": "bf16"},
        # the largest: a long prompt through the widest projection, short sums
        {"name": "gemm_long_prompt", "op": "gemm", "m": 8192, "n": 24576, "k": 1536, "fmt": "mxfp4", "dtype": "bf16"},
        # the step between two blocks of one sequence being generated
        {"name": "norm_one_token", "op": "norm", "m": 1, "k": 7168, "post": True, "gate": "none", "add": True,
         "offset": 0.0, "out": "same", "dtype": "bf16"},
        # the same step of a prompt: norm after the block, gate, residual, next norm into the FP8 linear's groups
        {"name": "norm_prompt_to_fp8", "op": "norm", "m": 4096, "k": 7168, "post": True, "gate": "sequence", "add": True,
         "offset": 1.0, "out": "fp8_128", "dtype": "bf16"},
        # a narrow norm by itself, odd in length
        {"name": "norm_narrow_odd", "op": "norm", "m": 8191, "k": 1536, "post": False, "gate": "none", "add": False,
         "offset": 0.0, "out": "same", "dtype": "fp16"},
        # a decode step of 16: gate, residual, norm into 4 bits, and the projection that reads them
        {"name": "linear_batch_16", "op": "linear", "m": 16, "n": 7168, "k": 2048, "fmt": "nvfp4", "source": "norm",
         "dtype": "bf16"},
        # a prompt's way out of a gated block: silu(gate) * up into 4 bits, and the product
        {"name": "linear_silu_prompt", "op": "linear", "m": 4096, "n": 7168, "k": 2048, "fmt": "mxfp4",
         "source": "silu", "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: max(work(c)["bytes"] + work(c)["flops"] / 1000 for c in listed() if c["op"] == op)
            for op in ("quant", "gemm", "norm", "linear")}
    while True:
        op = rng.choice(["quant", "gemm", "gemm", "gemm", "norm", "norm", "linear"])
        case = {"op": op, "m": _log_int(rng, 1, 8192), "dtype": rng.choice(["bf16", "fp16"])}
        fmt = rng.choice(["mxfp4", "nvfp4"])
        if op == "quant":
            case.update(k=_log_int(rng, 64, 16384) // 32 * 32, fmt=fmt, pad=rng.choice([0, 0, 64, 1024]))
        elif op == "gemm":
            case.update(n=_log_int(rng, 64, 24576) // 8 * 8, k=_log_int(rng, 64, 8192) // 32 * 32, fmt=fmt)
        elif op == "norm":
            out = rng.choice(["same", "same", "fp8_128", "fp8_32", "fp8_ue8m0_128", "fp8_ue8m0_32"])
            step = 8 if out == "same" else 128
            case.update(k=_log_int(rng, 128, 16384) // step * step, add=rng.random() < 0.7, offset=rng.choice([0.0, 1.0]),
                        out=out)
            case.update(post=case["add"] and rng.random() < 0.5,
                        gate=rng.choice(["none", "token", "sequence", "all"]) if case["add"] else "none")
        else:
            case.update(n=_log_int(rng, 64, 8192) // 8 * 8, k=_log_int(rng, 128, 8192) // 32 * 32, fmt=fmt,
                        source=rng.choice(["norm", "silu"]))
        w = work(case)
        if w["bytes"] + w["flops"] / 1000 <= most[op]:
            return case


def _packed(rows, k, fmt):
    return rows * k // 2 + rows * k // GROUP[fmt]


def _gate_rows(case):
    """Rows of the gate, each for as many consecutive tokens: one for all, one a sequence, one a token."""
    if case["gate"] == "all":
        return 1
    if case["gate"] == "sequence":
        return max(d for d in range(1, 9) if case["m"] % d == 0)
    return case["m"]


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quant":       # codes and scales written, and read again for the values
        return {"bytes": 4 * m * k + 2 * _packed(m, k, case["fmt"]), "flops": 4 * m * k}
    if op == "norm":
        rows = m * (1 + 2 * case["add"]) + (_gate_rows(case) if case["gate"] != "none" else 0)
        y = 2 * m * k if case["out"] == "same" else m * k + m * k // int(case["out"].split("_")[-1]) * (
            1 if "ue8m0" in case["out"] else 4)
        return {"bytes": 2 * k * rows + y + 2 * k * (1 + case["post"]), "flops": 10 * m * k}
    n = case["n"]
    product = _packed(n, k, case["fmt"]) + 2 * m * n
    if op == "gemm":
        return {"bytes": _packed(m, k, case["fmt"]) + product, "flops": 2 * m * n * k}
    into = 2 * m * k * (3 if case["source"] == "norm" else 2) + (2 * k * 2 if case["source"] == "norm" else 0)
    return {"bytes": into + 2 * _packed(m, k, case["fmt"]) + product, "flops": 2 * m * n * k + 10 * m * k}


# ---------------------------------------------------------------- the 4-bit form, with elementary operations

def _round_e2m1(q):
    """fp32 to the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code."""
    a = q.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, q)


def _encode(x, fmt, tensor_scale):
    """fp32 [m, k] -> (the codes' values [m, k], the groups' scales [m, k / group]), fp32."""
    g = GROUP[fmt]
    part = x.view(x.shape[0], -1, g)
    amax = part.abs().amax(dim=-1)
    if fmt == "mxfp4":
        half, e = torch.frexp(amax.clamp_min(1e-10) / 6.0)
        scale = torch.ldexp(torch.ones_like(half), e - (half == 0.5).int())
        whole = scale
    else:
        scale = (amax / (6.0 * tensor_scale)).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp_min(2.0 ** -9)
        whole = scale * tensor_scale
    return _round_e2m1(part / whole[..., None]).view_as(x), scale


def _values(codes, scale, fmt, tensor_scale):
    whole = scale if fmt == "mxfp4" else scale * tensor_scale
    return (codes.view(codes.shape[0], -1, GROUP[fmt]) * whole[..., None]).view_as(codes)


def _pack(codes, scale, fmt):
    """Codes two a byte, the even one low; scale bytes in tiles of 128 rows x 4 groups, byte
    (row % 32) * 16 + row / 32 * 4 + group of each tile's 512."""
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    nibble = torch.searchsorted(level, codes.abs()) + 8 * torch.signbit(codes)
    packed = (nibble[:, 0::2] + 16 * nibble[:, 1::2]).to(torch.uint8)
    byte = (torch.frexp(scale)[1] + 126).to(torch.uint8) if fmt == "mxfp4" else scale.to(torch.float8_e4m3fn).view(torch.uint8)
    rows, groups = byte.shape
    full = torch.zeros(-(-rows // 128) * 128, -(-groups // 4) * 4, dtype=torch.uint8, device=codes.device)
    full[:rows, :groups] = byte
    tiles = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return packed, tiles.reshape(tiles.shape[0], tiles.shape[1], 512).contiguous()


def _unpack(packed, tiles, fmt):
    """The other way: values of the codes and scales of the groups, fp32."""
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=packed.device)
    level = torch.cat([level, -level])
    rows, k = packed.shape[0], packed.shape[1] * 2
    codes = torch.stack([level[(packed & 15).int()], level[(packed >> 4).int()]], dim=-1).view(rows, k)
    byte = tiles.view(tiles.shape[0], tiles.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4)
    byte = byte.reshape(tiles.shape[0] * 128, -1)[:rows, :k // GROUP[fmt]].contiguous()
    if fmt == "mxfp4":
        return codes, torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.int() - 127)
    return codes, byte.view(torch.float8_e4m3fn).float()


# ---------------------------------------------------------------- inputs

def _scale_for(amax, fmt):
    """A tensor's scale in the two-level form: its largest value meets the largest code times the largest group scale."""
    return torch.full((1,), amax / (6.0 * 448.0), device="cuda") if fmt == "nvfp4" else None


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, m, k = DTYPES[case["dtype"]], case["m"], case["k"]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)

    def tensor(rows, std):
        """A tensor in the packed form, and its scale."""
        t = _scale_for(5.5 * std, case["fmt"])
        return (*_pack(*_encode(normal(rows, k, std=std).float(), case["fmt"], t), case["fmt"]), t)

    def wide(*shape):
        """Activations: a few channels are far larger than the others."""
        x = normal(*shape)
        loud = torch.randint(0, shape[-1], (max(1, shape[-1] // 1024),), generator=g, device="cuda")
        x[..., loud] *= 20
        return x

    s = {"case": case}
    if case["op"] == "quant":
        s["x"] = wide(m, k + case["pad"])[:, :k]
        s["scale"] = _scale_for(30 * math.pi, case["fmt"])     # calibrated ahead, on other data
    elif case["op"] == "gemm":
        s["a"], s["a_s"], s["a_t"] = tensor(m, 1.0)
        s["w"], s["w_s"], s["w_t"] = tensor(case["n"], 0.02)
    if case["op"] == "linear":
        s["w"], s["w_s"], s["w_t"] = tensor(case["n"], 0.02)
        s["a_t"] = _scale_for(12.0, case["fmt"])
        if case["source"] == "silu":
            s["x"] = normal(m, 2 * k)
    if case["op"] == "norm" or case.get("source") == "norm":
        add = case.get("add", True)
        s["x"] = wide(m, k)
        s["weight"] = normal(k, std=0.1, mean=1.0 - case.get("offset", 0.0))
        s["post"] = normal(k, std=0.1, mean=1.0 - case.get("offset", 0.0)) if case.get("post") else None
        s["residual"] = normal(m, k, std=3.0) if add else None
        s["gate"] = normal(_gate_rows(case), k, std=0.5) if case.get("gate", "none") != "none" else None
    return s


EPS, RESIDUAL, SCALE = 1e-6, 1.25, 0.5      # of the norms; how much of the residual and of the block's output is taken


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import fp8_block_scaled_sgq_gb300 as sgq

    case = s["case"]
    op, dtype, fmt = case["op"], DTYPES[case["dtype"]], case.get("fmt")
    if op == "quant":
        xq, xs = sgq.quant_fp4(s["x"], fmt, tensor_scale=s["scale"])
        return sgq.dequant_fp4(xq, xs, fmt, tensor_scale=s["scale"], dtype=dtype)
    if op == "gemm":
        return sgq.fp4_gemm(s["a"], s["a_s"], s["w"], s["w_s"], fmt, x_scale=s["a_t"], w_scale=s["w_t"], dtype=dtype)
    if op == "norm":
        quant, kw = None, {}
        if case["out"] != "same":
            quant, kw = case["out"].rsplit("_", 1)[0], {"group": int(case["out"].rsplit("_", 1)[1])}
        if not case["add"]:
            got = sgq.rms_norm(s["x"], s["weight"], eps=EPS, offset=case["offset"], quant=quant, **kw)
            got = got if quant else (got,)
        else:
            got = sgq.norm_add(s["x"], s["residual"], post_weight=s["post"], gate=s["gate"], scale=SCALE,
                               residual_scale=RESIDUAL, weight=s["weight"], eps=EPS, offset=case["offset"], quant=quant,
                               **kw)
        if quant is None:
            return got
        e8 = torch.float8_e8m0fnu if "ue8m0" in quant else torch.float32
        return (*got[:-2], got[-2].view(torch.float8_e4m3fn), got[-1].view(e8))
    if case["source"] == "silu":
        xq, xs = sgq.quant_fp4(s["x"], fmt, tensor_scale=s["a_t"], silu_mul=True)
        return sgq.fp4_gemm(xq, xs, s["w"], s["w_s"], fmt, x_scale=s["a_t"], w_scale=s["w_t"], dtype=dtype)
    h, xq, xs = sgq.norm_add(s["x"], s["residual"], scale=SCALE, residual_scale=RESIDUAL, weight=s["weight"], eps=EPS,
                             quant=fmt, tensor_scale=s["a_t"])
    return h, sgq.fp4_gemm(xq, xs, s["w"], s["w_s"], fmt, x_scale=s["a_t"], w_scale=s["w_t"], dtype=dtype)


def _norm(x, weight, offset):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * (weight.float() + offset)


def _plain_norm(s, dtype):
    """(the new residual in its type, or None, and the normed rows in fp32)"""
    case = s["case"]
    x, offset, h = s["x"].float(), case.get("offset", 0.0), None
    if s["residual"] is not None:
        if s["post"] is not None:
            x = _norm(x, s["post"], offset)
        if s["gate"] is not None:
            x = x * s["gate"].float().repeat_interleave(case["m"] // s["gate"].shape[0], dim=0)
        h = (RESIDUAL * s["residual"].float() + SCALE * x).to(dtype)
        x = h.float()
    return h, _norm(x, s["weight"], offset)


def _plain_product(a, a_s, a_t, s, fmt, dtype):
    """a, a_s: codes' values and scales of the activations."""
    w, w_s = _unpack(s["w"], s["w_s"], fmt)
    d = torch.matmul(_values(a, a_s, fmt, 1.0), _values(w, w_s, fmt, 1.0).T)
    return (d if fmt == "mxfp4" else d * (a_t * s["w_t"])).to(dtype)


def _run_plain(s):
    case = s["case"]
    op, dtype, fmt = case["op"], DTYPES[case["dtype"]], case.get("fmt")
    if op == "quant":
        return _values(*_encode(s["x"].float(), fmt, s["scale"]), fmt, s["scale"]).to(dtype)
    if op == "gemm":
        return _plain_product(*_unpack(s["a"], s["a_s"], fmt), s["a_t"], s, fmt, dtype)
    if op == "norm":
        h, y = _plain_norm(s, dtype)
        if case["out"] == "same":
            return (y.to(dtype),) if h is None else (h, y.to(dtype))
        g = int(case["out"].rsplit("_", 1)[1])
        scale = y.view(case["m"], -1, g).abs().amax(dim=-1).clamp_min(1e-10) / 448.0
        if "ue8m0" in case["out"]:
            half, e = torch.frexp(scale)
            scale = torch.ldexp(torch.ones_like(half), e - (half == 0.5).int())
        codes = (y.view(case["m"], -1, g) / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view_as(y)
        if "ue8m0" in case["out"]:
            scale = scale.to(torch.float8_e8m0fnu)
        return (codes, scale) if h is None else (h, codes, scale)
    if case["source"] == "silu":
        gate, up = s["x"].float().chunk(2, dim=-1)
        return _plain_product(*_encode(gate / (1.0 + torch.exp(-gate)) * up, fmt, s["a_t"]), s["a_t"], s, fmt, dtype)
    h, y = _plain_norm(s, dtype)
    return h, _plain_product(*_encode(y, fmt, s["a_t"]), s["a_t"], s, fmt, dtype)


# ---------------------------------------------------------------- the definition, in 64 bits

def _nearest(x, table):
    """The entry of a rising table of magnitudes that is nearest to |x|, ties to the even index, with x's sign."""
    mid = (table[1:] + table[:-1]) / 2
    low, high = torch.searchsorted(mid, x.abs(), right=False), torch.searchsorted(mid, x.abs(), right=True)
    return torch.copysign(table[torch.where(low % 2 == 0, low, high)], x)


def _tables():
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    code = torch.arange(127, dtype=torch.float64, device="cuda")            # 126 is 448, the largest
    e, f = torch.div(code, 8, rounding_mode="floor"), code % 8
    e4m3 = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7))
    return e2m1, e4m3


def _exact_quant(x, fmt, tensor_scale):
    """What quantisation to the format makes of x (64 bits)."""
    e2m1, e4m3 = _tables()
    part = x.unflatten(1, (-1, GROUP[fmt]))
    amax = part.abs().amax(dim=-1, keepdim=True)
    if fmt == "mxfp4":
        scale = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(1e-10) / 6)))
    else:
        t = tensor_scale.double()
        scale = _nearest((amax / (6 * t)).clamp(max=448), e4m3).clamp_min(2.0 ** -9) * t
    return (_nearest((part / scale).clamp(-6, 6), e2m1) * scale).flatten(1)


def _exact_values(packed, tiles, fmt):
    """Element by element: code and scale byte of (row, column) to their values."""
    e2m1, e4m3 = _tables()
    rows, k = packed.shape[0], 2 * packed.shape[1]
    out = torch.empty(rows, k, dtype=torch.float64, device="cuda")
    col = torch.arange(k, device="cuda")
    group = col // GROUP[fmt]
    for at in range(0, rows, 1024):
        r = torch.arange(at, min(at + 1024, rows), device="cuda")[:, None]
        nibble = (packed[r, col // 2].long() >> (4 * (col % 2))) & 15
        byte = tiles[r // 128, group // 4, r % 32 * 16 + r % 128 // 32 * 4 + group % 4].long()
        scale = torch.exp2(byte.double() - 127) if fmt == "mxfp4" else e4m3[byte]
        out[at:at + 1024] = e2m1[nibble & 7] * (1.0 - 2.0 * (nibble >> 3)) * scale
    return out


def _exact_product(x, s, fmt):
    d = x @ _exact_values(s["w"], s["w_s"], fmt).T
    return d if s["w_t"] is None else d * s["w_t"].double()


def exact(case, seed):
    if case["op"] in ("gemm", "linear") and 2.0 * case["m"] * case["n"] * case["k"] > 7e11:
        return None
    s = prepare(case, seed)
    op, fmt = case["op"], case.get("fmt")
    if op == "quant":
        return _exact_quant(s["x"].double(), fmt, s["scale"])
    if op == "gemm":
        x = _exact_values(s["a"], s["a_s"], fmt)
        return _exact_product(x if s["a_t"] is None else x * s["a_t"].double(), s, fmt)
    if case.get("source") == "silu":
        x = s["x"].double()
        y = x[:, :case["k"]] * torch.sigmoid(x[:, :case["k"]]) * x[:, case["k"]:]
        return _exact_product(_exact_quant(y, fmt, s["a_t"]), s, fmt)
    # the norms: each row over the root of its mean square
    k, offset = case["k"], case.get("offset", 0.0)
    h, y = None, s["x"].double()
    if s["residual"] is not None:
        if s["post"] is not None:
            y = y / (torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / k + EPS).sqrt() * (s["post"].double() + offset)
        if s["gate"] is not None:
            y = y * s["gate"].double()[torch.arange(case["m"], device="cuda") * s["gate"].shape[0] // case["m"]]
        h = s["residual"].double() * RESIDUAL + y * SCALE
        y = h.to(DTYPES[case["dtype"]]).double()        # the norm is of what is stored
    y = y / (torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / k + EPS).sqrt() * (s["weight"].double() + offset)
    if op == "linear":
        return h, _exact_product(_exact_quant(y, fmt, s["a_t"]), s, fmt)
    if case["out"] == "same":
        return (y,) if h is None else (h, y)
    _, e4m3 = _tables()
    part = y.unflatten(1, (-1, int(case["out"].rsplit("_", 1)[1])))
    scale = part.abs().amax(dim=-1).clamp_min(1e-10) / 448
    if "ue8m0" in case["out"]:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    codes = _nearest((part / scale[..., None]).clamp(-448, 448), e4m3).flatten(1)
    return (codes, scale) if h is None else (h, codes, scale)
