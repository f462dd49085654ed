"""What the operators of a server's decoder layer compute, on inputs of their real sizes.

A server runs many requests over one model at once.  Requests that begin with the same prompt
share its pages of the KV cache (``sink_attn_decode_shared`` reads them once for all); requests of
different customers share the projection's weights but bring their own low-rank adapters
(``lora_linear_bias`` adds them beside the product); and models with many small experts score them
with a softmax or a sigmoid, balance them with a bias and choose groups of experts first
(``moe_router_scores``).

Every case runs either in plain form (elementary torch operations, 32-bit arithmetic, 64 bits
where a choice between experts depends on it, rounded once at the end) or, with ``own`` set,
through this library's entry points.
"""
import math

import torch

own = False

PAGE, DIM, SM_SCALE = 16, 64, 0.125


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # four requests that have just begun on a prompt of 2048 tokens: latency counts
        {"name": "shared 4 x 2048", "op": "shared", "batch": 4, "groups": 1, "pages": 128, "own": 64, "hq": 64, "hkv": 8},
        # a decode step of 64 requests on one document of 32768 tokens
        {"name": "shared 64 x 32768", "op": "shared", "batch": 64, "groups": 1, "pages": 2048, "own": 1024, "hq": 64, "hkv": 8},
        # an odd batch in five groups of uneven prompts, query heads in groups of five
        {"name": "shared 37 in 5 groups", "op": "shared", "batch": 37, "groups": 5, "pages": 501, "own": 777, "hq": 40, "hkv": 8},
        # a full server: 512 requests on eight prompts, long answers
        {"name": "shared 512 in 8 groups", "op": "shared", "batch": 512, "groups": 8, "pages": 512, "own": 2048, "hq": 64, "hkv": 8},
        # output projection of one token with one adapter: latency
        {"name": "lora out, 1 token", "op": "lora", "tokens": 1, "k": 4096, "n": 2880, "rank": 16, "adapters": 8, "mix": "token"},
        # QKV projection of a decode step: nearly every request with an adapter of its own
        {"name": "lora qkv, 64 tokens", "op": "lora", "tokens": 64, "k": 2880, "n": 5120, "rank": 16, "adapters": 128, "mix": "token"},
        # output projection of a mixed step (short chunks and single tokens), some without adapter
        {"name": "lora out, 333 tokens", "op": "lora", "tokens": 333, "k": 4096, "n": 2880, "rank": 32, "adapters": 24, "mix": "chunk"},
        # QKV projection of a prefill batch: long runs of each request's tokens
        {"name": "lora qkv, 8192 tokens", "op": "lora", "tokens": 8192, "k": 2880, "n": 5120, "rank": 64, "adapters": 16, "mix": "prompt"},
        # router of a decode step: sigmoid scores, balance bias, 8 groups of experts, 4 of them kept
        {"name": "route 64 x 256", "op": "route", "tokens": 64, "experts": 256, "top_k": 8, "groups": 8, "keep": 4,
         "score": "sigmoid", "bias": True, "renorm": True, "type": "float32"},
        # softmax over all experts without groups, an odd number of tokens and of experts
        {"name": "route 4097 x 100", "op": "route", "tokens": 4097, "experts": 100, "top_k": 6, "groups": 1, "keep": 1,
         "score": "softmax", "bias": False, "renorm": False, "type": "bfloat16"},
        # a prefill batch of 4 x 8192 tokens
        {"name": "route 32768 x 256", "op": "route", "tokens": 32768, "experts": 256, "top_k": 8, "groups": 8, "keep": 4,
         "score": "sigmoid", "bias": True, "renorm": True, "type": "float32"},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "lora", "route"])
    if op == "shared":
        batch = _log_uniform(rng, 1, 512)
        hq, hkv = rng.choice([(64, 8), (32, 8), (40, 8), (28, 4), (16, 8), (8, 8), (32, 2)])
        pages = _log_uniform(rng, 1, 2048)
        if batch > 64:  # no more attention work than the fullest listed batch
            pages = min(pages, 512)
        return {"op": op, "batch": batch, "groups": rng.randint(1, min(8, batch)), "pages": pages,
                "own": _log_uniform(rng, 1, 2048), "hq": hq, "hkv": hkv}
    if op == "lora":
        k, n = 8 * rng.randint(16, 512), 8 * rng.randint(16, 640)
        tokens = _log_uniform(rng, 1, 8192)
        while tokens * k * n > 8192 * 2880 * 5120:
            k = max(128, k // 16 * 8)
        return {"op": op, "tokens": tokens, "k": k, "n": n, "rank": rng.choice([8, 16, 16, 24, 32, 64]),
                "adapters": rng.randint(1, 128), "mix": rng.choice(["token", "chunk", "prompt"])}
    groups = rng.choice([1, 1, 2, 4, 8])
    experts = groups * rng.randint(max(4, 8 // groups), 256 // groups)
    keep = rng.randint(1, groups)
    return {"op": op, "tokens": _log_uniform(rng, 1, 32768), "experts": experts,
            "top_k": rng.randint(1, min(8, keep * (experts // groups))), "groups": groups, "keep": keep,
            "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7,
            "type": rng.choice(["float32", "bfloat16"])}


def _layout(case):
    """Of a shared batch: where each group begins, its shared pages, and each request's length."""
    batch, groups = case["batch"], case["groups"]
    # uneven groups: weights 1, 2, 3, ... over the batch, at least one request each
    total = groups * (groups + 1) // 2
    starts = [g + (batch - groups) * (g * (g + 1) // 2) // total for g in range(groups)] + [batch]
    # uneven prompts: the first group has the longest; with more than two groups the last shares nothing
    pages = [max(1, case["pages"] * (2 * groups - g) // (2 * groups)) for g in range(groups)]
    if groups > 2:
        pages[-1] = 0
    lens = []
    for g in range(groups):
        for b in range(starts[g], starts[g + 1]):
            lens.append(PAGE * pages[g] + 1 + b * 7919 % case["own"])
    return starts, pages, lens


def work(case):
    op = case["op"]
    if op == "shared":
        starts, pages, lens = _layout(case)
        hq, hkv, batch = case["hq"], case["hkv"], case["batch"]
        own_tokens = sum(lens) - sum(PAGE * p * (starts[g + 1] - starts[g]) for g, p in enumerate(pages))
        tokens = PAGE * sum(pages) + own_tokens  # each shared page once, each request's own tokens once
        ids = 4 * (sum(pages) + own_tokens // PAGE + 2 * batch + 2 * case["groups"])
        return {"bytes": 4 * DIM * hkv * tokens + 4 * DIM * hq * batch + 4 * hq * (batch + 1) + ids,
                "flops": 4 * DIM * hq * sum(lens)}
    t = case["tokens"]
    if op == "lora":
        k, n, r, a = case["k"], case["n"], case["rank"], case["adapters"]
        # adapters that at least one of the runs of tokens picks (one run in eight has none)
        runs = len(_runs(case))
        active = round(a * (1 - (1 - 0.875 / a) ** runs))
        return {"bytes": 2 * (t * (k + n) + n * k + n + active * r * (k + n)) + 4 * (t + active),
                "flops": 2 * t * n * k + 2 * t * r * (k + n) * 7 // 8}
    size = 4 if case["type"] == "float32" else 2
    return {"bytes": t * (size * case["experts"] + 6 * case["top_k"]) + 4 * case["experts"] * case["bias"],
            "flops": 10 * t * case["experts"]}


def _runs(case):
    """Lengths of the runs of tokens that belong to one request."""
    t, runs, i = case["tokens"], [], 0
    while t:
        if case["mix"] == "token":
            n = 1
        elif case["mix"] == "chunk":  # every third a chunk, the others single tokens
            n = 1 if i % 3 else 1 + (i * 37 + 16) % 61
        else:
            n = max(1, case["tokens"] // 5 + (i * 271) % 97 - 48)
        n = min(n, t)
        runs.append(n)
        t -= n
        i += 1
    return runs


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, op = {"case": case}, case["op"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * std).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    if op == "shared":
        starts, pages, lens = _layout(case)
        hq, hkv, batch = case["hq"], case["hkv"], case["batch"]
        width = max((n + PAGE - 1) // PAGE for n in lens)
        first_own, used = [], sum(pages)
        for grp, p in enumerate(pages):
            for b in range(starts[grp], starts[grp + 1]):
                first_own.append(used)
                used += (lens[b] + PAGE - 1) // PAGE - p
        # pages lie anywhere in the cache, as a server's allocator leaves them
        place = torch.randperm(used, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
        done = 0
        for grp, p in enumerate(pages):
            for b in range(starts[grp], starts[grp + 1]):
                table[b, :p] = place[done : done + p]
                own_pages = (lens[b] + PAGE - 1) // PAGE - p
                table[b, p : p + own_pages] = place[first_own[b] : first_own[b] + own_pages]
            done += p
        s.update(q=normal(batch, hq, DIM), k=normal(used, hkv, PAGE, DIM), v=normal(used, hkv, PAGE, DIM), table=table,
                 lens=ints(lens), starts=ints(starts), pages=ints(pages), sinks=normal(hq, dtype=torch.float32),
                 host=(starts, pages, lens), max_pages=max(pages))
    elif op == "lora":
        k, n, r, a, t = case["k"], case["n"], case["rank"], case["adapters"], case["tokens"]
        runs = _runs(case)
        pick = torch.randint(0, a, (len(runs),), generator=g, device="cuda")
        none = torch.rand(len(runs), generator=g, device="cuda") < 0.125
        pick = torch.where(none, -1, pick).to(torch.int32)
        s["adapter"] = pick.repeat_interleave(torch.tensor(runs, device="cuda"))
        s["present"] = sorted(set(pick.tolist()) - {-1})
        s.update(x=normal(t, k), w=normal(n, k, std=1 / math.sqrt(k)), bias=normal(n),
                 a=normal(a, r, k, std=1 / math.sqrt(k)), b=normal(a, n, r, std=1 / math.sqrt(r)),
                 scale=0.25 + 0.75 * torch.rand(a, generator=g, device="cuda"))
    else:
        t, e = case["tokens"], case["experts"]
        # some experts are asked for more often; the bias works against that
        liking = 0.5 * torch.randn(e, generator=g, device="cuda")
        logits = 1.5 * torch.randn(t, e, generator=g, device="cuda") + liking
        s["logits"] = logits.to(getattr(torch, case["type"]))
        s["bias"] = -0.1 * liking + 0.01 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
    torch.cuda.synchronize()
    return s


# ----------------------------------------------------------------------------- plain forms
def _matmul(a, b, operands_are_bf16):
    """a b in fp32.  bf16 values have 8 significant bits, so the tensor cores' 11-bit operands
    hold them exactly and only the fp32 sums round; other operands stay in 32 bits."""
    torch.backends.cuda.matmul.allow_tf32 = operands_are_bf16
    return a @ b


def _plain_shared(s):
    starts, pages, lens = s["host"]
    case = s["case"]
    hq, hkv = case["hq"], case["hkv"]
    grp = hq // hkv
    outs, lses = [], []
    for g, p in enumerate(pages):
        b0, b1 = starts[g], starts[g + 1]
        n = b1 - b0
        q = s["q"][b0:b1].float().reshape(n, hkv, grp, DIM)
        parts = [s["sinks"].reshape(1, hkv, grp, 1).expand(n, hkv, grp, 1)]
        values = []
        if p:
            ids = s["table"][b0, :p].long()
            k = s["k"][ids].permute(1, 0, 2, 3).reshape(hkv, p * PAGE, DIM).float()
            values.append(s["v"][ids].permute(1, 0, 2, 3).reshape(hkv, p * PAGE, DIM).float())
            x = _matmul(q.permute(1, 0, 2, 3).reshape(hkv, n * grp, DIM), k.mT, True) * SM_SCALE
            parts.append(x.reshape(hkv, n, grp, p * PAGE).transpose(0, 1))
        own = max(lens[b0:b1]) - p * PAGE  # the own parts, padded to the longest
        own_pages = (own + PAGE - 1) // PAGE
        ids = s["table"][b0:b1, p : p + own_pages].long()
        k = s["k"][ids].permute(0, 2, 1, 3, 4).reshape(n, hkv, own_pages * PAGE, DIM).float()
        v = s["v"][ids].permute(0, 2, 1, 3, 4).reshape(n, hkv, own_pages * PAGE, DIM).float()
        x = _matmul(q, k.mT, True) * SM_SCALE
        seen = torch.arange(own_pages * PAGE, device=x.device) < (s["lens"][b0:b1, None] - p * PAGE)
        parts.append(x.masked_fill(~seen[:, None, None], -math.inf))
        top = torch.stack([t.amax(-1) for t in parts]).amax(0).unsqueeze(-1)
        e = [torch.exp(t - top) for t in parts]
        z = sum(t.sum(-1, keepdim=True) for t in e)
        o = _matmul(e[-1], v, False)
        if p:
            y = e[1].transpose(0, 1).reshape(hkv, n * grp, p * PAGE)
            o = o + _matmul(y, values[0], False).reshape(hkv, n, grp, DIM).transpose(0, 1)
        outs.append((o / z).reshape(n, hq, DIM).to(torch.bfloat16))
        lses.append((top + torch.log(z)).reshape(n, hq))
    return torch.cat(outs), torch.cat(lses)


def _plain_lora(s):
    x = s["x"].float()
    y = _matmul(x, s["w"].float().T, True) + s["bias"].float()
    case = s["case"]
    if case["tokens"] * case["rank"] * max(case["k"], case["n"]) <= 1 << 28:  # every token's own adapter, as a batch
        at = s["adapter"].clamp(min=0).long()
        t = _matmul(s["a"][at].float(), x.unsqueeze(2), True) * (s["scale"][at] * (s["adapter"] >= 0)).reshape(-1, 1, 1)
        return (y + _matmul(s["b"][at].float(), t, False).squeeze(2)).to(torch.bfloat16)
    for a in s["present"]:
        rows = (s["adapter"] == a).nonzero().reshape(-1)
        t = _matmul(x[rows], s["a"][a].float().T, True) * s["scale"][a]
        y.index_add_(0, rows, _matmul(t, s["b"][a].float().T, False))
    return y.to(torch.bfloat16)


def _plain_route(s):
    case = s["case"]
    t, e, groups = case["tokens"], case["experts"], case["groups"]
    x = s["logits"].double()  # values next to a border decide between experts
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        z = torch.exp(x - x.amax(1, keepdim=True))
        score = z / z.sum(1, keepdim=True)
    value = score if s["bias"] is None else score + s["bias"].double()
    if case["keep"] < groups:
        by_group = value.reshape(t, groups, e // groups)
        merit = by_group.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        kept = merit.sort(dim=1, descending=True, stable=True).indices[:, : case["keep"]]
        inside = torch.zeros(t, groups, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        value = by_group.masked_fill(~inside.unsqueeze(2), -math.inf).reshape(t, e)
    idx = value.sort(dim=1, descending=True, stable=True).indices[:, : case["top_k"]]
    w = score.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (2.5 * w).to(torch.bfloat16)


def _plain(s):
    return {"shared": _plain_shared, "lora": _plain_lora, "route": _plain_route}[s["case"]["op"]](s)


# ----------------------------------------------------------------------------- the library's calls
def _own(s):
    import attention_softmax_sinks_gb300 as sa

    case = s["case"]
    if case["op"] == "shared":
        return sa.sink_attn_decode_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["sinks"], s["starts"], s["pages"],
                                          s["max_pages"], SM_SCALE)
    if case["op"] == "lora":
        return sa.lora_linear_bias(s["x"], s["w"], s["a"], s["b"], s["adapter"], bias=s["bias"], lora_scale=s["scale"])
    return sa.moe_router_scores(s["logits"], case["top_k"], score=case["score"], bias=s["bias"], num_groups=case["groups"],
                                top_groups=case["keep"], renormalize=case["renorm"], scale=2.5)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "shared":
        starts, pages, lens = s["host"]
        grp = case["hq"] // case["hkv"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):  # request by request, over its whole cache
            ids = s["table"][b, : (n + PAGE - 1) // PAGE].long()
            k = s["k"][ids].double().transpose(0, 1).flatten(1, 2)[:, :n]
            v = s["v"][ids].double().transpose(0, 1).flatten(1, 2)[:, :n]
            x = torch.einsum("hgd,hnd->hgn", s["q"][b].double().unflatten(0, (-1, grp)), k).flatten(0, 1) * SM_SCALE
            x = torch.cat([x, s["sinks"].double()[:, None]], 1)
            lse[b] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b][:, None])[:, :n]
            out[b] = torch.einsum("hgn,hnd->hgd", p.unflatten(0, (-1, grp)), v).flatten(0, 1)
        return out, lse
    if case["op"] == "lora":
        y = s["bias"].double() + s["x"].double() @ s["w"].double().T
        ids = s["adapter"].tolist()
        first = 0
        while first < len(ids):  # run by run
            last = first
            while last < len(ids) and ids[last] == ids[first]:
                last += 1
            if ids[first] >= 0:
                a = ids[first]
                y[first:last] += s["scale"][a].double() * ((s["x"][first:last].double() @ s["a"][a].double().T) @ s["b"][a].double().T)
            first = last
        return y
    # the weights of the experts; which ones is a whole number and has to be equal
    x = s["logits"].double()
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    value = score + (0 if s["bias"] is None else s["bias"].double())
    e, groups = case["experts"], case["groups"]
    if case["keep"] < groups:
        best = torch.topk(value.unflatten(1, (groups, -1)), 2, dim=2).values.sum(2)
        # a group stays if fewer than `keep` others come before it
        before = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & torch.ones(
            groups, groups, dtype=torch.bool, device="cuda").tril(-1))
        value = torch.where((before.sum(2) < case["keep"]).repeat_interleave(e // groups, 1), value, -math.inf)
    rest, picked = value.clone(), []
    for _ in range(case["top_k"]):  # one expert after the other; argmax of equal values: the first
        top = rest.amax(1, keepdim=True)
        at = torch.where(rest == top, torch.arange(e, device="cuda"), e).amin(1, keepdim=True)
        picked.append(score.gather(1, at))
        rest = rest.scatter(1, at, -math.inf)
    w = torch.cat(picked, 1)
    return None, 2.5 * (w / w.sum(1, keepdim=True) if case["renorm"] else w)
