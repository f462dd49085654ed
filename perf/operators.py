"""What the expert layer's operators compute, on inputs of their real sizes.

Behind the router, a mixture-of-experts layer sorts its (token, expert) pairs by expert
(``moe_group_rows``), runs each expert's two matrix products on its ragged group of rows
(``grouped_linear_swiglu`` / ``grouped_linear_bias`` in bf16, ``grouped_mxfp4_linear_*`` on
4-bit operands), and adds each token's expert outputs up again (``moe_combine``).  4-bit
operands come from ``mxfp4_quantize``; ``mxfp4_linear_bias`` is the product of one matrix.

Every case runs either in plain form (elementary torch operations, 32-bit arithmetic,
rounded once at the end) or, with ``own`` set, through this library's entry points.
"""
import math

import torch

own = False

ALPHA, LIMIT = 1.702, 7.0  # SwiGLU constants of the public GPT-OSS configuration
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # the routing of one decode step of 64 sequences, and of the 4 x 8192-token prefill batch
        {"name": "group decode 64", "op": "group", "tokens": 64, "experts": 128, "top_k": 4},
        {"name": "group prefill 32768", "op": "group", "tokens": 32768, "experts": 128, "top_k": 4},
        # gate and up projection of one token: four experts' weights are streamed once
        {"name": "experts up, 1 token", "op": "experts", "tokens": 1, "experts": 128, "top_k": 4,
         "k": 2880, "n": 5760, "act": "swiglu", "gather": True},
        # down projection of an odd decode batch: nearly every expert has one or two rows
        {"name": "experts down, 61 tokens", "op": "experts", "tokens": 61, "experts": 128, "top_k": 4,
         "k": 2880, "n": 2880, "act": "none", "gather": False},
        # gate and up projection of the 4 x 8192-token prefill batch: bound by the tensor cores
        {"name": "experts up, 32768 tokens", "op": "experts", "tokens": 32768, "experts": 128, "top_k": 4,
         "k": 2880, "n": 5760, "act": "swiglu", "gather": True},
        # activations of a decode step and of the prefill batch, before a 4-bit product
        {"name": "mxfp4 quantize 64", "op": "quantize", "tokens": 64, "k": 2880, "type": "bfloat16"},
        {"name": "mxfp4 quantize 32768", "op": "quantize", "tokens": 32768, "k": 2880, "type": "bfloat16"},
        # the QKV projection of a prefill chunk on 4-bit operands
        {"name": "mxfp4 linear 8192", "op": "mxfp4", "tokens": 8192, "experts": 0, "top_k": 1,
         "k": 2880, "n": 5120, "act": "none", "gather": False},
        # the two gate and up projections above on 4-bit operands
        {"name": "mxfp4 experts up, 1 token", "op": "mxfp4", "tokens": 1, "experts": 128, "top_k": 4,
         "k": 2880, "n": 5760, "act": "swiglu", "gather": True},
        {"name": "mxfp4 experts up, 32768 tokens", "op": "mxfp4", "tokens": 32768, "experts": 128, "top_k": 4,
         "k": 2880, "n": 5760, "act": "swiglu", "gather": True},
        # the experts' outputs of a decode step and of the prefill batch, added up per token
        {"name": "combine decode 64", "op": "combine", "tokens": 64, "k": 2880, "top_k": 4},
        {"name": "combine prefill 32768", "op": "combine", "tokens": 32768, "k": 2880, "top_k": 4},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "experts", "experts", "quantize", "mxfp4", "mxfp4", "combine"])
    tokens = _log_uniform(rng, 1, 32768)
    experts = rng.choice([8, 31, 32, 64, 100, 128])
    top_k = rng.choice([1, 2, 4, 4, 6, 8])
    if op == "group":
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k}
    if op == "quantize":
        return {"op": op, "tokens": tokens, "k": 32 * rng.randint(2, 90), "type": rng.choice(["bfloat16", "float32"])}
    if op == "combine":
        return {"op": op, "tokens": tokens, "k": 8 * rng.randint(8, 360), "top_k": rng.choice([1, 2, 4])}
    # products: inputs and features up to the listed ones, at most the largest case's rows
    k, n = 32 * rng.randint(2, 90), 2 * rng.randint(32, 2880)
    if op == "mxfp4" and rng.random() < 0.25:
        return {"op": op, "tokens": min(tokens, 8192), "experts": 0, "top_k": 1, "k": k, "n": min(n, 5120),
                "act": "none", "gather": False}
    tokens = max(1, min(tokens, 131072 // top_k))
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "k": k, "n": n,
            "act": rng.choice(["swiglu", "none"]), "gather": rng.choice([True, False])}


def work(case):
    t, op = case["tokens"], case["op"]
    if op == "group":  # the indices once; offsets, the rows' tokens and the pairs' rows once
        pairs = t * case["top_k"]
        return {"bytes": 4 * (3 * pairs + case["experts"] + 1), "flops": 0}
    if op == "quantize":  # read the values, write codes and scales, read them again, write the values
        size, blocks = (4 if case["type"] == "float32" else 2), t * case["k"] // 32
        return {"bytes": blocks * (32 * size + 2 * 17 + 32 * 2), "flops": 0}
    if op == "combine":
        pairs = t * case["top_k"]
        return {"bytes": 2 * case["k"] * (pairs + t) + 6 * pairs, "flops": 2 * pairs * case["k"]}
    rows, k, n = t * case["top_k"], case["k"], case["n"]
    e = case["experts"]
    # experts that at least one of t tokens picks, each token picking top_k of e evenly
    active = round(e * (1 - (1 - case["top_k"] / e) ** t)) if e else 1
    out = rows * (n // 2 if case["act"] == "swiglu" else n)
    x_rows = t if case["gather"] else rows
    per_value = 17 / 32 if op == "mxfp4" else 2  # 4-bit codes and a scale byte for 32 of them
    total = per_value * k * (x_rows + active * n) + 2 * active * n + 2 * out
    if e:
        total += 4 * (e + 1) + (4 * rows if case["gather"] else 0)
    return {"bytes": total, "flops": 2 * rows * n * k}


# ----------------------------------------------------------------------------- inputs
def _routing(g, tokens, experts, top_k):
    """Expert choices as a router makes them: some experts are asked for more often."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda") + 0.3 * torch.randn(experts, generator=g, device="cuda")
    return logits.topk(min(top_k, experts), dim=1).indices.to(torch.int32)


def _pack(values, exponents):
    """E2M1 values and their blocks' exponents as codes (two per byte, the first in the low
    half) and scale bytes (rows padded with zeros to a multiple of 16)."""
    mag = values.abs()
    code = ((mag >= 0.5).to(torch.uint8) + (mag >= 1.0) + (mag >= 1.5) + (mag >= 2.0) + (mag >= 3.0) + (mag >= 4.0) + (mag >= 6.0))
    code = (code + 8 * (values < 0)).to(torch.uint8)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = (exponents + 127).to(torch.uint8)
    return codes.contiguous(), torch.nn.functional.pad(scales, (0, -scales.shape[-1] % 16)).contiguous()


def _mxfp4_operand(g, shape, std):
    """A matrix (or a stack of them) of normal values in MXFP4, one matrix at a time."""
    out = [_pack(*_to_fp4(std * torch.randn(shape[-2:], generator=g, device="cuda"))) for _ in range(math.prod(shape[:-2]))]
    codes, scales = (torch.stack(v).reshape(*shape[:-1], -1) for v in zip(*out))
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, t = case["op"], case["tokens"]
    s = {"case": case}

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * std).to(dtype)

    if op == "group":
        s["topk_idx"] = _routing(g, t, case["experts"], case["top_k"])
    elif op == "quantize":
        # activations: blocks of very different size, a few outliers, some zeros
        x = torch.randn(t, case["k"], generator=g, device="cuda")
        x = x * torch.exp(1.5 * torch.randn(t, case["k"] // 32, generator=g, device="cuda")).repeat_interleave(32, 1)
        x = torch.where(torch.rand(t, case["k"], generator=g, device="cuda") < 0.01, torch.zeros_like(x), x)
        s["x"] = x.to(getattr(torch, case["type"]))
    elif op == "combine":
        pairs = t * case["top_k"]
        s["y"] = normal(pairs, case["k"])
        s["pair_row"] = torch.randperm(pairs, generator=g, device="cuda").to(torch.int32).reshape(t, case["top_k"])
        s["weight"] = torch.randn(t, case["top_k"], generator=g, device="cuda").softmax(1).to(torch.bfloat16)
    else:
        k, n, e = case["k"], case["n"], case["experts"]
        std = 1.0 / math.sqrt(k)
        if e:
            # the plan a program keeps between the router and the products
            idx = _routing(g, t, e, case["top_k"])
            flat = idx.reshape(-1).long()
            counts = torch.bincount(flat, minlength=e)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            if case["gather"]:
                s["row_token"] = (flat.argsort(stable=True) // idx.shape[1]).to(torch.int32)
            s["active"] = counts.nonzero().reshape(-1)
            s["longest"] = int(counts.max())
            rows = t if case["gather"] else flat.numel()
        else:
            rows = t
        lead = (e,) if e else ()
        s["bias"] = normal(*lead, n)
        if op == "mxfp4":
            s["x"], s["x_scales"] = _mxfp4_operand(g, (rows, k), 1.0)
            s["w"], s["w_scales"] = _mxfp4_operand(g, (*lead, n, k), std)
        else:
            s["x"] = normal(rows, k)
            s["w"] = normal(e, n, k, std=std)
    torch.cuda.synchronize()
    return s


# ----------------------------------------------------------------------------- plain forms
def _power_of_two(exponent):
    """2^exponent in fp32, exactly, for exponents from -127 (a subnormal number) to 127."""
    normal = ((exponent.clamp(min=-126) + 127).to(torch.int32) << 23).view(torch.float32)
    return torch.where(exponent < -126, 2.0 ** -127, normal)


def _to_fp4(x):
    """Blocks of 32 scaled by 2^(floor(log2 of the largest magnitude) - 2), rounded to the
    nearest E2M1 value (ties to even, at most 6): values and block exponents."""
    blocks = x.float().reshape(*x.shape[:-1], -1, 32)
    largest = blocks.abs().amax(-1)
    exponent = torch.where(largest > 0, torch.frexp(largest).exponent - 3, -127).clamp(-127, 125)
    v = blocks * _power_of_two(-exponent).unsqueeze(-1)
    mag = v.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(mag / step) * step).clamp(max=6.0), v)
    return q.reshape(x.shape), exponent


def _from_codes(codes, scales):
    """The fp32 values of MXFP4 codes and scale bytes (exact: two significant bits each)."""
    pairs = torch.tensor([[FP4[b & 15], FP4[b >> 4]] for b in range(256)], device=codes.device)
    v = torch.nn.functional.embedding(codes.int(), pairs).flatten(-2)
    blocks = v.unflatten(-1, (-1, 32))
    return (blocks * _power_of_two(scales[..., : blocks.shape[-2]].int() - 127).unsqueeze(-1)).flatten(-2)


def _product(x, w, bias):
    """x w^T + bias in fp32.  bf16 and MXFP4 values have at most 8 significant bits, so the
    tensor cores' 11-bit operands hold them exactly and only the fp32 sums round."""
    torch.backends.cuda.matmul.allow_tf32 = True
    return x @ w.mT + bias.float()


def _swiglu(y):
    gate, up = y[..., 0::2].clamp(max=LIMIT), y[..., 1::2].clamp(-LIMIT, LIMIT)
    return gate * torch.sigmoid(ALPHA * gate) * (up + 1)


def _plain_experts(s, x, w):
    """Every group that has rows, padded to the longest, as one batched product."""
    offsets, active = s["offsets"].long(), s["active"]
    total = x.shape[0] if "row_token" not in s else s["row_token"].shape[0]
    rows = offsets[active][:, None] + torch.arange(s["longest"], device=x.device)
    inside = rows < offsets[active + 1][:, None]
    source = rows.clamp(max=total - 1)
    if "row_token" in s:
        source = s["row_token"].long()[source]
    y = _product(x[source], w, s["bias"][active][:, None])
    if s["case"]["act"] == "swiglu":
        y = _swiglu(y)
    out = torch.empty(total + 1, y.shape[-1], dtype=torch.bfloat16, device=x.device)
    out[torch.where(inside, rows, total)] = y.to(torch.bfloat16)  # what is padding goes to the row behind
    return out[:total]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "group":
        idx, e = s["topk_idx"], case["experts"]
        flat = idx.reshape(-1).long()
        order = flat.argsort(stable=True)
        counts = torch.zeros(e, dtype=torch.int64, device=idx.device).scatter_add_(0, flat, torch.ones_like(flat))
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        pair_row = torch.empty_like(flat)
        pair_row[order] = torch.arange(flat.numel(), device=idx.device)
        return offsets.int(), (order // idx.shape[1]).int(), pair_row.reshape(idx.shape).int()
    if op == "quantize":
        q, exponent = _to_fp4(s["x"])
        return (q.unflatten(-1, (-1, 32)) * _power_of_two(exponent).unsqueeze(-1)).flatten(-2).to(torch.bfloat16)
    if op == "combine":
        return (s["weight"].float().unsqueeze(-1) * s["y"][s["pair_row"].long()].float()).sum(1).to(torch.bfloat16)
    if op == "experts":
        return _plain_experts(s, s["x"].float(), s["w"][s["active"]].float())
    x = _from_codes(s["x"], s["x_scales"])
    if not case["experts"]:
        return _product(x, _from_codes(s["w"], s["w_scales"]), s["bias"]).to(torch.bfloat16)
    return _plain_experts(s, x, _from_codes(s["w"][s["active"]], s["w_scales"][s["active"]]))


# ----------------------------------------------------------------------------- the library's calls
def _own(s):
    import attention_softmax_sinks_gb300 as sa

    case, op = s["case"], s["case"]["op"]
    if op == "group":
        return sa.moe_group_rows(s["topk_idx"], case["experts"])
    if op == "quantize":
        return sa.mxfp4_dequantize(*sa.mxfp4_quantize(s["x"]))
    if op == "combine":
        return sa.moe_combine(s["y"], s["pair_row"], s["weight"])
    swiglu, rows = case["act"] == "swiglu", s.get("row_token")
    if op == "experts":
        if swiglu:
            return sa.grouped_linear_swiglu(s["x"], s["w"], s["offsets"], s["bias"], row_token=rows, alpha=ALPHA, limit=LIMIT)
        return sa.grouped_linear_bias(s["x"], s["w"], s["offsets"], s["bias"], row_token=rows)
    if not case["experts"]:
        return sa.mxfp4_linear_bias(s["x"], s["x_scales"], s["w"], s["w_scales"], s["bias"])
    if swiglu:
        return sa.grouped_mxfp4_linear_swiglu(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"], s["bias"],
                                              row_token=rows, alpha=ALPHA, limit=LIMIT)
    return sa.grouped_mxfp4_linear_bias(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"], s["bias"], row_token=rows)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- in 64 bits
def _fp64_of_codes(codes, scales):
    table = torch.tensor(FP4, dtype=torch.float64, device=codes.device)
    nibbles = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    blocks = nibbles.shape[-1] // 32
    power = ((scales[..., :blocks].long() - 127 + 1023) << 52).view(torch.float64)
    return table[nibbles.long()] * power.repeat_interleave(32, -1)


def exact(case, seed):
    op = case["op"]
    if op == "group":
        return None  # whole numbers
    if op in ("experts", "mxfp4") and work(case)["flops"] > 6e12:
        return None  # fp64 products of this size take too long
    s = prepare(case, seed)
    if op == "quantize":
        # the nearest of the eight magnitudes, found by comparison with each
        x = s["x"].double().reshape(-1, 32)
        # the double's own exponent field holds floor(log2); a zero has -1023 there
        power = ((x.abs().amax(1, keepdim=True).view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)
        scale = ((power + 1023) << 52).view(torch.float64)
        grid = torch.tensor(FP4[:8], dtype=torch.float64, device=x.device)
        best, away = torch.zeros_like(x), torch.full_like(x, math.inf)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they win ties
            d = (x.abs() / scale - grid[i]).abs()
            best, away = torch.where(d < away, grid[i], best), torch.minimum(d, away)
        return (torch.sign(x) * best * scale).reshape(s["x"].shape)
    if op == "combine":
        out = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device="cuda")
        for r in range(case["top_k"]):
            out += s["weight"][:, r : r + 1].double() * s["y"].index_select(0, s["pair_row"][:, r]).double()
        return out
    wide = (lambda name, at: _fp64_of_codes(s[name][at], s[name + "_scales"][at])) if op == "mxfp4" else (lambda name, at: s[name][at].double())
    if not case["experts"]:
        return wide("x", slice(None)) @ wide("w", slice(None)).T + s["bias"].double()
    ends = s["offsets"].tolist()
    parts = []
    for e in range(case["experts"]):
        if ends[e] == ends[e + 1]:
            continue
        at = slice(ends[e], ends[e + 1]) if not case["gather"] else s["row_token"][ends[e] : ends[e + 1]].long()
        y = wide("x", at) @ wide("w", e).T + s["bias"][e].double()
        if case["act"] == "swiglu":
            gate, up = y[:, 0::2], y[:, 1::2]
            gate, up = torch.clamp(gate, max=LIMIT), torch.clamp(up, min=-LIMIT, max=LIMIT)
            y = (up + 1) * gate / (1 + torch.exp(-ALPHA * gate))
        parts.append(y)
    return torch.cat(parts)
