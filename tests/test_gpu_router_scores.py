"""Router by scores, groups and balance, against the definition in 64 bits.

The experts have to be equal.  Weights: the score in fp32 is off by less than 2^-19 relative
(exp2 and reciprocal 2^-22 each, the exponent's rounding 2^-24 |x| for |x| <= 16, sums of 256), the
sum for renormalising as much again, and the rounding to bf16 by 2^-8: 2^-8 + 2^-17 of the weight."""
import pytest
import torch

pytestmark = pytest.mark.gpu
INF = float("inf")


def make(t, e, dtype="float32", bias=None, std=1.5, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (std * torch.randn(t, e, generator=g, device="cuda")).to(getattr(torch, dtype))
    b = None if bias is None else bias * torch.randn(e, generator=g, device="cuda")
    return x, b


def two_sum(x, y):
    """x + y without rounding, as a sum of two doubles (adding a huge bias must not hide a score)."""
    s = x + y
    z = s - x
    e = (x - (s - z)) + (y - z)
    return s, torch.where(torch.isfinite(s), e, 0.0)


def descending(hi, lo):
    """Indices of hi + lo, largest first, equal ones in order."""
    first = lo.sort(dim=-1, descending=True, stable=True).indices
    return first.gather(-1, hi.gather(-1, first).sort(dim=-1, descending=True, stable=True).indices)


def reference(x, k, score, bias, groups, keep, renorm, scale):
    x = x.double()
    t, e = x.shape
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    v, v2 = two_sum(s, torch.zeros(e, dtype=torch.float64, device="cuda") if bias is None else bias.double())
    idx = descending(x, torch.zeros_like(x)) if bias is None else descending(v, v2)  # without bias: the logits' order
    if keep < groups:
        g, g2 = v.reshape(t, groups, -1), v2.reshape(t, groups, -1)
        two = descending(g, g2)[:, :, :2]
        g, g2 = g.gather(2, two), g2.gather(2, two).sum(2)
        m, m2 = two_sum(g[:, :, 0], g[:, :, 1]) if two.shape[2] == 2 else (g[:, :, 0], torch.zeros_like(g2))
        kept = descending(*two_sum(m, m2 + g2))[:, :keep]
        inside = torch.zeros(t, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        out = ~inside.repeat_interleave(e // groups, 1).gather(1, idx)
        idx = idx.gather(1, out.int().sort(dim=1, stable=True).indices)
    idx = idx[:, :k]
    w = s.gather(1, idx)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return idx, scale * w


def check(x, k, score="softmax", bias=None, groups=1, keep=1, renorm=True, scale=1.0, **kw):
    import attention_softmax_sinks_gb300 as sa
    idx, w, counts = sa.moe_router_scores(x, k, score=score, bias=bias, num_groups=groups, top_groups=keep,
                                          renormalize=renorm, scale=scale, return_counts=True, **kw)
    ri, rw = reference(x, k, score, bias, groups, keep, renorm, scale)
    wrong = (idx.long() != ri).any(1)
    assert not bool(wrong.any()), f"{int(wrong.sum())} tokens differ, first {int(wrong.nonzero()[0])}: {idx[wrong][0].tolist()} {ri[wrong][0].tolist()}"
    assert bool(((w.double() - rw).abs() <= (2.0 ** -8 + 2.0 ** -17) * rw.abs() + 1e-38).all())
    assert torch.equal(counts.long(), torch.bincount(ri.reshape(-1), minlength=x.shape[1]))


SHAPES = [(1, 256, 8, 8, 4), (3, 1, 1, 1, 1), (64, 256, 8, 8, 4), (5, 7, 3, 1, 1), (130, 100, 6, 4, 2), (33, 160, 6, 8, 3),
          (1000, 64, 4, 1, 1), (17, 255, 8, 5, 5), (40, 96, 2, 32, 7), (9, 32, 8, 32, 8), (31, 60, 5, 20, 10),
          (20, 256, 7, 2, 1), (700, 128, 1, 16, 3), (12, 200, 8, 8, 1), (50, 31, 8, 31, 9)]


@pytest.mark.parametrize("t,e,k,groups,keep", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("bias", [None, 0.1])
def test_router_scores(t, e, k, groups, keep, score, dtype, bias):
    x, b = make(t, e, dtype, bias, seed=e + k)
    check(x, k, score, b, groups, keep, renorm=(t % 2 == 0), scale=1.0 if t % 3 else 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 4)])
@pytest.mark.parametrize("bias", [None, 0.05])
def test_many_tokens(score, groups, keep, bias):
    # some of 200000 tokens have neighbours that fp32 cannot tell apart
    x, b = make(200000, 256, "float32", bias, seed=7)
    check(x, 8, score, b, groups, keep)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_values(score):
    # bf16 logits from a handful of values, and a bias of few values: ties everywhere
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randint(-3, 4, (3000, 128), generator=g, device="cuda") / 2).to(torch.bfloat16)
    for bias in (None, torch.zeros(128, device="cuda"), torch.randint(0, 2, (128,), generator=g, device="cuda") / 8.0):
        check(x, 8, score, bias)
        check(x, 6, score, bias, 8, 3)
    same = torch.zeros(5, 256, device="cuda")
    check(same, 8, score, None, 8, 2)
    check(same, 8, score, torch.zeros(256, device="cuda"), 16, 16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbouring_floats(score):
    # logits one step of fp32 apart: no score in 32 bits tells them apart
    base = torch.tensor(0.7, device="cuda")
    steps = torch.arange(64, device="cuda", dtype=torch.int32)
    row = (base.view(torch.int32) + steps).view(torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.stack([row[torch.randperm(64, generator=g, device="cuda")] for _ in range(200)])
    check(x, 8, score)
    check(x, 8, score, None, 4, 2)
    check(x, 8, score, 1e-8 * torch.randn(64, generator=g, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1e-6, 30.0, 1e4, 1e30])
def test_biases_of_any_size(score, size):
    x, b = make(500, 96, "float32", size, seed=5)
    check(x, 8, score, b)
    check(x, 4, score, b, 6, 2)
    check(x, 8, score, torch.full((96,), size, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_at_the_extremes(score):
    x, b = make(300, 64, std=3.0, seed=9)
    x[:, 5] = -INF
    x[1, :60] = -INF        # four experts left for eight places
    x[2] = x[2] * 25        # far below the largest: scores that vanish in fp32
    x[3] = 80 + x[3]        # sigmoids that round to one
    x[4] = -80 + x[4]
    for bias in (None, b):
        check(x[:2], 8, score, bias, renorm=False) if score == "sigmoid" or bias is None else None
    check(x, 8, score)
    check(x, 4, score, None, 8, 8)
    import attention_softmax_sinks_gb300 as sa
    out = torch.full((3, 64), -INF, device="cuda")  # nothing to choose from: the first experts, without weight
    idx, w = sa.moe_router_scores(out, 8, score=score)
    assert torch.equal(idx.cpu(), torch.arange(8, dtype=torch.int32).repeat(3, 1)) and bool((w == 0).all())


def test_disabled_experts():
    x, b = make(100, 64, seed=2)
    bias = torch.zeros(64, device="cuda")
    bias[::2] = -INF
    check(x, 8, "sigmoid", bias)
    check(x, 8, "softmax", bias, 4, 2)


def test_not_a_number_stays_in_range():
    import attention_softmax_sinks_gb300 as sa
    x, b = make(64, 256, seed=4)
    x[::2, ::3] = float("nan")
    x[1] = float("nan")
    x[3, :9] = INF
    for bias in (None, torch.randn(256, device="cuda"), torch.full((256,), float("nan"), device="cuda"),
                 torch.where(torch.arange(256, device="cuda") % 7 == 0, INF, 0.0)):
        for groups, keep in ((1, 1), (8, 3)):
            idx, _ = sa.moe_router_scores(x, 8, "sigmoid", bias, groups, keep)
            assert bool(((idx >= 0) & (idx < 256)).all())


def test_unaligned_rows():
    base = torch.randn(50 * 64 + 3, device="cuda")
    for off in (1, 2, 3):
        check(base[off : off + 50 * 64].reshape(50, 64), 4, "sigmoid", None, 4, 2)
    half = base.to(torch.bfloat16)
    for off in (1, 2, 3):
        check(half[off : off + 50 * 64].reshape(50, 64), 4)


def test_no_tokens():
    import attention_softmax_sinks_gb300 as sa
    idx, w, c = sa.moe_router_scores(torch.empty(0, 64, device="cuda"), 4, return_counts=True)
    assert idx.shape == (0, 4) and bool((c == 0).all())


def test_outputs_stream_and_graph():
    import attention_softmax_sinks_gb300 as sa
    x, b = make(500, 256, bias=0.1)
    args = dict(score="sigmoid", bias=b, num_groups=8, top_groups=4, scale=2.5)
    want = sa.moe_router_scores(x, 8, **args)
    idx = torch.full((510, 8), -9, dtype=torch.int32, device="cuda")
    w = torch.full((510, 8), -9.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sa.moe_router_scores(x, 8, **args, topk_idx=idx[:500], topk_weight=w[:500], stream=s)
    s.synchronize()
    assert torch.equal(idx[:500], want[0]) and torch.equal(w[:500], want[1])
    assert bool((idx[500:] == -9).all()) and bool((w[500:] == -9).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gi, gw, gc = sa.moe_router_scores(x, 8, **args, return_counts=True)
    x.copy_(make(500, 256, seed=8)[0])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    ri, rw = reference(x, 8, "sigmoid", b, 8, 4, True, 2.5)
    assert torch.equal(gi.long(), ri) and torch.equal(gc.long(), torch.bincount(ri.reshape(-1), minlength=256))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_that_share_a_huge_bias(score):
    x, _ = make(300, 64, seed=6)
    bias = torch.zeros(64, device="cuda")
    bias[7::5] = 1e20
    check(x, 8, score, bias)
    check(x, 6, score, bias, 8, 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [-INF, torch.finfo(torch.float32).min, -3e38, -1e9, -1e4])
def test_groups_with_one_expert_left(score, mask):
    # a merit is the sum of two values: a masked one takes it below those of groups with two others
    x = torch.tensor([[3.0, 3.0, -1.0, -1.0]], device="cuda")
    check(x, 1, score, torch.tensor([0.0, mask, 0.0, 0.0], device="cuda"), 2, 1)
    x, bias = make(400, 64, bias=0.1, seed=21)
    e = torch.arange(64, device="cuda")
    for size in (2, 4, 8):
        group = e // size
        masked = ((group % 3 == 0) & (e % size > 0)) | (group % 5 == 1)  # one left of some groups, none of others
        b = torch.where(masked, mask, bias)
        groups = 64 // size
        for keep in (1, groups // 3, groups // 2, groups - 1):  # the last: groups with one or none are kept, too
            check(x, min(6, keep * size), score, b, groups, keep)
    # groups of one expert
    x, e, bias = x[:, :32].contiguous(), e[:32], bias[:32]
    check(x, 5, score, torch.where(e % 2 == 0, mask, bias), 32, 7)
    check(x, 8, score, torch.where(e % 4 != 0, mask, bias), 32, 9)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_are_ordered_as_well(score):
    # fewer experts left than places: the masked ones follow by their values, equal ones by index
    x, bias = make(200, 64, bias=0.1, seed=22)
    e = torch.arange(64, device="cuda")
    low = torch.finfo(torch.float32).min
    for mask in (low, -1e9, -1e4, -INF):
        check(x, 8, score, torch.where(e % 13 == 5, bias, mask))
        check(x, 8, score, torch.where(e % 9 == 0, bias, mask), 8, 2)
    mixed = torch.where(e % 4 == 0, -INF, torch.where(e % 4 == 1, low, torch.where(e % 4 == 2, -1e5, bias)))
    check(x, 8, score, mixed)
    check(x, 8, score, torch.where(e > 20, mixed.clamp(max=-1e5), bias))
    check(x, 6, score, mixed, 16, 5)
    check(x, 8, score, mixed.roll(3), 8, 3)
    check(x, 8, score, torch.full((64,), low, device="cuda"))
    check(x, 8, score, torch.where(e == 9, 1e4, bias))          # one far above the others
    check(x, 4, score, torch.where(e == 9, 1e4, bias), 8, 3)
    check(x, 8, score, torch.where(e < 9, 3e38, -3e38))         # their distance is beyond fp32
    check(x, 4, score, torch.where(e % 2 == 0, 3e38, -3e38), 8, 3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_pinned_by_an_infinite_bias(score):
    x, bias = make(200, 64, bias=0.1, seed=23)
    x[:, 9] = -4.0  # not for its score
    bias[9] = INF
    check(x, 1, score, bias)
    check(x, 8, score, bias)
    check(x, 8, score, bias, 8, 3)
    bias[[2, 40, 41]] = INF
    check(x, 3, score, bias)
    check(x, 6, score, bias, 16, 5)
    bias[20:40] = -INF
    check(x, 8, score, bias)
    check(x, 8, score, bias, 8, 7)
    check(x, 8, score, torch.full((64,), INF, device="cuda"))


@pytest.mark.parametrize("lanes", [1, 2, 8])
def test_sum_of_many_small_exponentials(lanes):
    # Terms of the softmax's sum that are each below half a step of the largest one, but not together:
    # the largest score and another expert's bias are the same to within a few 2^-24.
    x = torch.full((512, 256), -100.0, device="cuda")
    small = [4 * (j + 8 * i) + c for j in range(lanes) for i in range(8) for c in range(4)]
    small += [e for e in (5, 9, 17) if e not in small]
    small = [e for e in small if e not in (0, 23)]
    x[:, small] = torch.linspace(-16.6362, -16.8, 512, device="cuda")[:, None]
    x[:, 0] = 0.0
    exact = torch.softmax(x.double(), 1)[:, 0]
    for at in (0, 100, 300, 511):
        for away in range(-4, 5):
            bias = torch.zeros(256, device="cuda")
            bias[23] = exact[at] + away * 2.0 ** -25
            check(x, 1, "softmax", bias)
            check(x, 2, "softmax", bias, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_equal_neighbours_do_not_hide_a_third(score, dtype):
    # scores that no key tells apart: the border's two experts have the same logit, a later one a larger
    zero = torch.zeros(32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(24)
    for base, more in ((20.0, 0.5), (30.0, 1.0), (0.0, 1e-7), (-50.0, 0.25)):
        x = torch.full((64, 32), base, device="cuda")
        x[:, 31] = 5.0 if base < 5.0 else 100.0  # the largest, for what is relative to it
        at = torch.randint(3, 31, (64, 2), generator=g, device="cuda")
        x.scatter_(1, at, base + more)
        x = x.to(getattr(torch, dtype))
        for k in (1, 2, 3, 4, 8):
            for bias in (None, zero, zero - 0.75):
                check(x, k, score, bias)
            check(x, k, score, None, 4, 2)
            check(x, k, score, zero, 4, 3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_whose_mask_leaves_nothing(score):
    # every logit -inf: the scores are 0 and the biases decide, also where they are nearly the same
    import attention_softmax_sinks_gb300 as sa
    g = torch.Generator(device="cuda").manual_seed(25)
    x = torch.randn(6, 64, generator=g, device="cuda")
    x[::2] = -INF
    order = torch.randperm(64, generator=g, device="cuda").float()
    for step in (2.0 ** -25, 2.0 ** -22, 2.0 ** -10):
        bias = 0.25 + order * step
        for k, groups, keep in ((8, 1, 1), (3, 1, 1), (6, 8, 3), (8, 32, 5)):
            idx, w = sa.moe_router_scores(x, k, score=score, bias=bias, num_groups=groups, top_groups=keep)
            ri, _ = reference(x[::2], k, "sigmoid", bias, groups, keep, True, 1.0)  # whose score of -inf is 0
            assert torch.equal(idx[::2].long(), ri)
            assert bool((w[::2] == 0).all())
            ri, rw = reference(x[1::2], k, score, bias, groups, keep, True, 1.0)
            assert torch.equal(idx[1::2].long(), ri)


def test_infinite_logits_by_sigmoid():
    x, bias = make(300, 64, bias=0.1, seed=26)
    x[:, 40] = INF
    x[1::3, 50:] = INF
    x[2::3, :30] = -INF
    for b in (None, bias):
        for k in (1, 3, 8):
            check(x, k, "sigmoid", b)
        check(x, 6, "sigmoid", b, 8, 3)
        check(x[:, :32].contiguous(), 5, "sigmoid", None if b is None else b[:32].contiguous(), 32, 7)
    check(x.to(torch.bfloat16), 8, "sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [torch.finfo(torch.float32).min, -1e9, -1e3])
def test_pinned_and_masked_experts_in_one_group(score, mask):
    # +inf and a finite mask make a merit of +inf, as +inf and any other bias
    x, bias = make(200, 64, bias=0.1, seed=27)
    e = torch.arange(64, device="cuda")
    bias = torch.where((e // 4 % 4 == 1) & (e % 4 != 2), mask, bias)
    bias[[0, 6, 22, 33, 34]] = INF
    for groups in (16, 8, 32):
        for keep in (1, 2, 3, 5, 7):
            check(x, 2, score, bias, groups, keep)
            check(x, min(8, 64 // groups * keep), score, bias, groups, keep)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 4)])
@pytest.mark.parametrize("std", [0.002, 1.5, 12.0])
def test_many_equal_logits_in_bf16(score, groups, keep, std):
    x, b = make(20000, 256, "bfloat16", 0.05, std=std, seed=8)
    for bias in (None, b, b.to(torch.bfloat16).float() * 0.0):
        for k in (1, 8):
            check(x, k, score, bias, groups, keep)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_chosen_scores_that_vanish_in_fp32(score, dtype):
    # a bias chooses experts far below the largest: their weights add up to scale all the same
    x, _ = make(300, 64, dtype, std=3.0, seed=28)
    bias = torch.zeros(64, device="cuda")
    bias[8:] = -2.0
    bias[3] = -1.5
    x[:, 8:] += 60
    for below in (0.0, 40.0, 90.0, 130.0, 300.0):
        y = x.clone()
        y[:, :8] -= below
        y[::7, 2:8] = -INF
        y[5, :8] = -INF
        for k, groups, keep in ((4, 1, 1), (8, 1, 1), (3, 8, 1), (8, 16, 3)):
            check(y, k, score, bias, groups, keep, scale=2.5)
            check(y, k, score, bias, groups, keep, renorm=False)
    check((x - 500).clamp(max=-100), 8, score)
