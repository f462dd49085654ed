"""One layer of a decode step with the operators a server would run behind one another: products with
adapters around the attention of a batch that shares prompts, the router by scores and the experts
behind it.  Each step is held to its own formula in 64 bits on the inputs that it got (so that a
rounding before it cannot change what it has to choose); the whole run, captured and replayed,
alone and beside another one, gives the same bits again."""
import threading

import pytest
import torch

import test_gpu_lora as lora
import test_gpu_router_scores as scores
import test_gpu_shared as shared

pytestmark = pytest.mark.gpu
PAGE, DIM = 16, 64
SA_OK, SA_ERR_TIMEOUT = 0, 6


def layer(groups, own, hq=16, hkv=2, hid=512, inner=128, experts=32, adapters=5, rank=16, seed=0):
    """A layer's weights, a batch's cache and its new tokens' values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(c for c, _ in groups)

    def normal(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)

    def product(n_out, n_in):
        return dict(w=normal(n_out, n_in, std=n_in ** -0.5), lora_a=normal(adapters, rank, n_in, std=n_in ** -0.5),
                    lora_b=normal(adapters, n_out, rank, std=rank ** -0.5), bias=normal(n_out),
                    lora_scale=torch.randn(adapters, generator=g, device="cuda"))

    attn = shared.make(groups, own, hq, hkv, seed=seed + 1)
    del attn["q"]
    for name in ("paged_k", "paged_v"):  # the new tokens' rows are written by the run itself
        attn[name] = attn[name].nan_to_num(0.0)
    return dict(x=normal(n, hid), idx=torch.tensor(lora.mixed(n, adapters, seed), dtype=torch.int32, device="cuda"),
                qkv=product((hq + 2 * hkv) * DIM, hid), o=product(hid, hq * DIM), attn=attn, hq=hq,
                cu=torch.arange(n + 1, dtype=torch.int32, device="cuda"), router=normal(experts, hid, std=hid ** -0.5),
                balance=0.1 * torch.randn(experts, generator=g, device="cuda"), up=normal(experts, 2 * inner, hid, std=hid ** -0.5),
                down=normal(experts, hid, inner, std=inner ** -0.5), experts=experts)


def run(sa, l, stream=None):
    """The layer's steps; every step's result."""
    r = {}
    a = l["attn"]
    r["qkv"] = sa.lora_linear_bias(l["x"], adapter_idx=l["idx"], stream=stream, **l["qkv"])
    r["q"] = sa.qkv_bias_rope_append_paged(r["qkv"], None, l["cu"], a["kv_lens"], a["paged_k"], a["paged_v"], a["page_table"],
                                           l["hq"], stream=stream)
    r["attn"], r["lse"] = sa.sink_attn_decode_shared(r["q"], stream=stream, **a)
    r["y"] = sa.lora_linear_bias(r["attn"].view(len(r["attn"]), -1), adapter_idx=l["idx"], stream=stream, **l["o"])
    r["logits"] = sa.linear_bias(r["y"], l["router"], stream=stream)
    r["experts"], r["weights"] = sa.moe_router_scores(r["logits"], 4, "sigmoid", l["balance"], 8, 3, scale=2.5, stream=stream)
    off, tok, row = sa.moe_group_rows(r["experts"], l["experts"], stream=stream)
    h = sa.grouped_linear_swiglu(r["y"], l["up"], off, row_token=tok, stream=stream)
    r["rows"] = sa.grouped_linear_bias(h, l["down"], off, stream=stream)
    r["out"] = sa.moe_combine(r["rows"], row, r["weights"], stream=stream)
    return r


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


BATCHES = {
    "three groups": ([(9, 6), (14, 17), (1, 0)], [1 + 37 * i % 300 for i in range(24)]),
    "one token, one sequence": ([(1, 3)], [1]),
    "one long prompt": ([(40, 300)], [1 + 29 * i % 200 for i in range(40)]),
    "one prompt": ([(70, 40)], [1 + 11 * i % 90 for i in range(70)]),
}


@pytest.mark.parametrize("name", BATCHES)
def test_steps_of_a_layer(name):
    import attention_softmax_sinks_gb300 as sa
    sa.sink_attn_device_status(True)
    l = layer(*BATCHES[name], seed=3)
    r = run(sa, l)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 0
    lora.check(dict(x=l["x"], adapter_idx=l["idx"], **l["qkv"]), r["qkv"])
    shared.check(dict(q=r["q"], **l["attn"]), r["attn"], r["lse"])
    lora.check(dict(x=r["attn"].view(len(r["attn"]), -1), adapter_idx=l["idx"], **l["o"]), r["y"])
    ri, rw = scores.reference(r["logits"], 4, "sigmoid", l["balance"], 8, 3, True, 2.5)
    assert torch.equal(r["experts"].long(), ri)
    assert bool(((r["weights"].double() - rw).abs() <= (2.0 ** -8 + 2.0 ** -17) * rw).all())
    # the weights in bf16 are what the experts' rows are added up with
    off, _, row = sa.moe_group_rows(r["experts"], l["experts"])
    assert torch.equal(off[-1].long(), torch.tensor(4 * len(r["y"]), device="cuda"))
    rows = r["rows"].double()[row.long()]
    want = (r["weights"].double()[:, :, None] * rows).sum(1)
    mag = (r["weights"].double()[:, :, None] * rows).abs().sum(1)
    assert bool(((r["out"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 4 * 2.0 ** -24 * mag + 1e-30).all())
    # the plain decode, which reads every sequence's pages for itself
    a = {k: v for k, v in l["attn"].items() if k not in ("group_offsets", "shared_pages", "max_shared_pages")}
    plain, plain_lse = sa.sink_attn_decode(r["q"], **a)
    _, _, mag = shared.reference(dict(q=r["q"], **l["attn"]))
    assert bool(((plain.double() - r["attn"].double()).abs() <= 2.0 ** -7 * (r["attn"].double().abs() + mag) + 2.0 ** -12 * mag).all())
    assert bool(((plain_lse - r["lse"]).abs() <= 2.0 ** -12 + 2.0 ** -21 * r["lse"].abs()).all())


def test_captured_replayed_and_beside_another():
    """Two layers captured as graphs that allocate what they need, replayed alone and at the same time
    on two streams, with other tokens in the same places; and from two threads without graphs."""
    import attention_softmax_sinks_gb300 as sa
    sa.sink_attn_device_status(True)
    ls = [layer(*BATCHES["three groups"], seed=5), layer(*BATCHES["one long prompt"], seed=6)]
    eager = [{k: v.clone() for k, v in run(sa, l).items()} for l in ls]
    streams = [torch.cuda.Stream() for _ in ls]
    graphs, results = [], []
    for l, s in zip(ls, streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            results.append(run(sa, l))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(e, r) for e, r in zip(eager, results))
    # other tokens, other adapters, in the same memory
    for l in ls:
        l["x"].copy_(l["x"].flip(0))
        l["idx"].copy_(l["idx"].roll(1))
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    changed = [{k: v.clone() for k, v in r.items()} for r in results]
    again = [run(sa, l) for l in ls]
    torch.cuda.synchronize()
    assert all(same(c, r) for c, r in zip(changed, again))
    assert not same(changed[0], eager[0])
    got, errors, start = [None, None], [], threading.Barrier(2)

    def work(i):
        try:
            torch.cuda.set_device(0)
            s = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got[i] = run(sa, ls[i], stream=s)
            s.synchronize()
        except Exception as e:  # reported after the join
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not errors, errors
    torch.cuda.synchronize()
    assert all(same(c, r) for c, r in zip(changed, got))
    assert sa.sink_attn_device_status(True) == 0


def test_zero_wait_budget_unwinds_cleanly():
    """Under a zero budget waits may give up at once; the kernels then drain their copies and
    products, free TMEM and report, and the next call is right."""
    import attention_softmax_sinks_gb300 as sa
    sa.sink_attn_device_status(True)
    a = shared.make([(40, 200), (3, 30)], [1 + 7 * i for i in range(43)], 16, 2)
    few = lora.make(64, 2880, 1280, 16, 9, lora.mixed(64, 9))
    many = lora.make(2000, 2880, 2560, 16, 5, [(i // 370) % 5 for i in range(2000)])
    try:
        sa.sink_attn_set_wait_timeout_ns(0)
        sa.sink_attn_decode_shared(**a)
        sa.lora_linear_bias(**few)
        sa.lora_linear_bias(**many)
        assert sa.sink_attn_device_status(True) in (SA_OK, SA_ERR_TIMEOUT)
    finally:
        sa.sink_attn_set_wait_timeout_ns(2_000_000_000)
    shared.check(a, *shared.call(a))
    for b in (few, many):
        lora.check(b, lora.call(b))
