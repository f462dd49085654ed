"""Linear layer with low-rank adapters, against the formula in 64 bits.

Tolerances.  Products of bf16 values are exact in fp32; the tensor cores sum K of them in fp32,
off by at most K 2^-23 of the sum of magnitudes (truncation allowed).  With t = x A^T:
  t            K 2^-23 sum |x a|, its parts' sum 4 * 2^-24 more: dt
  s t in bf16  2^-8 |s t| and one fp32 rounding, |s| dt
  out          (K + R + 1) 2^-23 (sum |x w| + |bias| + sum |s t b|), the errors of s t times |b|,
               and 2^-8 |out| for the rounding to bf16."""
import pytest
import torch

pytestmark = pytest.mark.gpu
NAN = float("nan")


def make(m, k, n, r, l, idx, bias=True, scale=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)

    return dict(x=normal(m, k), w=normal(n, k, std=k ** -0.5), lora_a=normal(l, r, k, std=k ** -0.5),
                lora_b=normal(l, n, r, std=r ** -0.5), adapter_idx=torch.tensor(idx, dtype=torch.int32, device="cuda"),
                bias=normal(n) if bias else None,
                lora_scale=torch.randn(l, generator=g, device="cuda") if scale else None)


def reference(a):
    """out and its error bound, in 64 bits."""
    x, w = a["x"].double(), a["w"].double()
    (m, k), n, r = x.shape, w.shape[0], a["lora_a"].shape[1]
    b = a["bias"].double() if a["bias"] is not None else torch.zeros(n, dtype=torch.float64, device="cuda")
    out, mag = x @ w.T + b, x.abs() @ w.abs().T + b.abs()
    err = torch.zeros_like(out)
    for i in set(a["adapter_idx"].tolist()):
        if i < 0 or i >= a["lora_a"].shape[0]:
            continue
        rows = (a["adapter_idx"] == i).nonzero().reshape(-1)
        la, lb = a["lora_a"][i].double(), a["lora_b"][i].double()
        s = a["lora_scale"][i].double() if a["lora_scale"] is not None else 1.0
        st = s * (x[rows] @ la.T)
        dt = abs(s) * (k + 4) * 2.0 ** -23 * (x[rows].abs() @ la.abs().T)
        out[rows] += st @ lb.T
        mag[rows] += st.abs() @ lb.abs().T
        err[rows] += (dt + (2.0 ** -8 + 2.0 ** -20) * st.abs()) @ lb.abs().T
    return out, err + (k + r + 1) * 2.0 ** -23 * mag + 2.0 ** -8 * out.abs()


def check(a, out):
    ref, bound = reference(a)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), f"worst error / bound {(err / bound).nan_to_num(1e9).max().item()}"


def call(a, **kw):
    import attention_softmax_sinks_gb300 as sa
    sa.sink_attn_device_status(True)
    out = sa.lora_linear_bias(**a, **kw)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 0
    return out


def mixed(m, l, seed=1, none=0.2):
    g = torch.Generator().manual_seed(seed)
    pick = torch.randint(0, l, (m,), generator=g)
    return torch.where(torch.rand(m, generator=g) < none, -1, pick).tolist()


CASES = {
    "one token": (1, 256, 64, 16, 3, [2]),
    "one token, smallest": (1, 8, 8, 8, 1, [0]),
    "one token, no adapter": (1, 64, 72, 16, 3, [-1]),
    "nobody has an adapter": (300, 128, 200, 32, 4, [-1] * 300),
    "rank 8": (70, 200, 120, 8, 5, mixed(70, 5)),
    "rank 24": (33, 328, 248, 24, 7, mixed(33, 7)),
    "rank 32": (128, 512, 512, 32, 9, mixed(128, 9)),
    "rank 40": (129, 512, 136, 40, 3, mixed(129, 3)),
    "rank 64": (257, 640, 264, 64, 4, mixed(257, 4)),
    "rank 72": (100, 136, 328, 72, 40, mixed(100, 40)),
    "rank 128": (200, 1000, 400, 128, 6, mixed(200, 6)),
    "every token its own": (128, 264, 96, 16, 128, list(range(127, -1, -1))),
    "every token its own, rank 128": (128, 72, 72, 128, 200, list(range(0, 128))),
    "most adapters": (300, 64, 72, 16, 1024, [(i * 331) % 1024 for i in range(300)]),
    "one adapter for all": (700, 384, 640, 16, 2, [1] * 700),
    "runs": (1000, 320, 512, 64, 5, [(i // 170) % 5 for i in range(1000)]),
    "long K": (5, 6144, 256, 16, 4, [0, 1, 1, -1, 3]),
    "tall": (20000, 64, 96, 16, 8, [(i // 999) % 8 for i in range(20000)]),
    "wide": (3, 64, 40000, 16, 2, [0, 1, -1]),
    "decode, 64 tokens": (64, 2880, 5120, 16, 128, mixed(64, 128)),
    "clusters, 100 tokens": (100, 2880, 1000, 32, 60, mixed(100, 60)),
    "clusters, odd sizes": (7, 1032, 4104, 24, 9, mixed(7, 9)),
    "clusters, two row blocks": (200, 4096, 1032, 64, 90, mixed(200, 90)),
    "clusters, rank 128": (61, 2880, 2880, 128, 61, list(range(61))),
    "pairs, runs": (2700, 264, 5120, 64, 5, [(i // 370) % 5 for i in range(2700)]),
    "pairs, mixed": (2049, 128, 5000, 16, 300, mixed(2049, 300)),
    "pairs, rank 128": (2304, 200, 4352, 128, 3, mixed(2304, 3)),
    "pairs, rank 24": (5000, 72, 2880, 24, 40, mixed(5000, 40)),
}


@pytest.mark.parametrize("name", CASES)
def test_lora_linear(name):
    m, k, n, r, l, idx = CASES[name]
    a = make(m, k, n, r, l, idx, seed=len(name))
    check(a, call(a))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scale", [False, True])
def test_without_bias_or_scale(bias, scale):
    a = make(90, 256, 328, 16, 5, mixed(90, 5), bias=bias, scale=scale)
    check(a, call(a))


def test_without_adapters_like_linear_bias():
    import attention_softmax_sinks_gb300 as sa
    a = make(333, 1024, 520, 16, 5, [-1] * 333)
    # the sums' order differs (parts of K): each result is within the bound, so they differ by twice it
    got, want = call(a), sa.linear_bias(a["x"], a["w"], a["bias"])
    assert bool(((got.double() - want.double()).abs() <= 2 * reference(a)[1]).all())


def test_tokens_stand_alone():
    # a token's result does not depend on who shares its tile; unused adapters may hold anything
    a = make(130, 512, 264, 32, 16, mixed(130, 15))
    a["lora_a"][15], a["lora_b"][15] = NAN, NAN
    out = call(a)
    for m in (0, 57, 129):
        one = {**a, "x": a["x"][m : m + 1].contiguous(), "adapter_idx": a["adapter_idx"][m : m + 1].contiguous()}
        got, want = call(one).double(), out[m : m + 1].double()
        assert bool(((got - want).abs() <= 2 * reference(one)[1]).all())


def test_not_finite_stays_with_its_tokens():
    a = make(20, 128, 72, 16, 4, [i % 4 for i in range(20)])
    a["lora_b"][2, 5, 3] = NAN
    a["x"][7, 3] = float("inf")  # a token of adapter 3
    out = call(a).float()
    bad = ~torch.isfinite(out)
    expect = torch.zeros_like(bad)
    expect[2::4, 5] = True
    expect[7] = True
    assert torch.equal(bad, expect)


def test_bad_index_is_reported():
    import attention_softmax_sinks_gb300 as sa
    a = make(40, 128, 72, 16, 4, [i % 4 for i in range(40)])
    a["adapter_idx"][11], a["adapter_idx"][12] = 4, 2 ** 31 - 1
    out = sa.lora_linear_bias(**a)
    torch.cuda.synchronize()
    assert sa.sink_attn_device_status(True) == 5
    check(a, out)


def test_outputs_workspace_and_stream():
    import attention_softmax_sinks_gb300 as sa
    a = make(140, 512, 264, 16, 9, mixed(140, 9))
    want = call(a)
    need = sa.lora_workspace_bytes(140, 512, 16)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((150, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sa.lora_linear_bias(**a, workspace=ws, out=out[:140], stream=s)
    s.synchronize()
    assert torch.equal(got, want) and bool((out[140:] == 7).all()) and bool((ws[need:] == 255).all())


def test_repeated_calls_and_graph_replay():
    import attention_softmax_sinks_gb300 as sa
    a = make(300, 512, 1024, 16, 9, mixed(300, 9))
    want = call(a)
    for _ in range(5):
        assert torch.equal(call(a), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sa.lora_linear_bias(**a)
        out2 = sa.lora_linear_bias(**{**a, "x": out[:, :512].contiguous()})
    b = make(300, 512, 1024, 16, 9, mixed(300, 9, seed=4), seed=3)
    for name in a:
        a[name].copy_(b[name])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    check(a, out)
    check({**a, "x": out[:, :512].contiguous()}, out2)
    assert sa.sink_attn_device_status(True) == 0


@pytest.mark.parametrize("name", ["one token", "rank 24", "rank 128", "runs", "decode, 64 tokens", "clusters, odd sizes",
                                  "clusters, two row blocks", "pairs, mixed", "pairs, rank 128", "pairs, rank 24"])
def test_rows_and_adapters_that_are_not_finite(name):
    # rows of NaN (what pads a batch), infinite ones, adapters with a NaN in either factor: each row as by itself
    m, k, n, r, l, idx = CASES[name]
    a = make(m, k, n, r, l, idx, seed=len(name))
    inf = float("inf")
    if m > 1:
        a["x"][0] = NAN
        a["adapter_idx"][0] = -1
        a["x"][m // 2, k // 3] = NAN
        a["x"][m // 3, 5] = inf
        a["x"][-1, 0], a["x"][-1, 1] = inf, -inf
    used = sorted(set(a["adapter_idx"].tolist()) - {-1})
    a["lora_b"][used[0], 7, 3] = NAN
    a["lora_b"][used[-1], n - 1, 0] = inf
    if len(used) > 2:
        a["lora_b"][used[1]] = NAN
        a["lora_a"][used[2], 1, 2] = NAN
    out = call(a).double()
    ref, bound = reference(a)
    good = torch.isfinite(ref)
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    assert torch.equal(torch.isfinite(out), good) and torch.equal(out[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert bool(((out - ref).abs() <= bound)[good].all())
